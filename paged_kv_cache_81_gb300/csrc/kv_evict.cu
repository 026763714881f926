// kv_evict: trims every request to the tokens that weigh most.
//
// Of a request with more than `budget` tokens the first `sinks`, the last `recent` and, of the others, the
// ones of highest score stay (equal scores: lowest index first), in their order; their rows in every
// tensor and plane are gathered to the request's first `budget` slots of the output table.
//
// evict_select_kernel, a CTA per request: a radix select over the scores' bits, eleven at a time (scores
// mapped to unsigned integers of the same order), finds the key of the last token that stays and how many
// equal ones stay; one more pass in index order writes the list, its position coming from one block scan
// of (above, equal) counts.  evict_move_kernel, bound by memory: a CTA walks a stretch of the list for a
// (request, tensor, plane) in chunks of 32 KB, all loads of a chunk before its stores.  In place, slot i
// receives a row of slot >= i, so chunks in order never overwrite a row that is still to be read.  16 requests
// of 4000 to 16000 tokens trimmed to 2048 in 32 tensors of 8 x 128 take 673 us, 94% of the copy rate (851 in
// place, where one CTA walks a whole list); four short ones in two tensors 9.9 us, most of it the two launches' latencies.
#include <algorithm>

#include "kv_attention.cuh"

namespace pkv {

namespace {

constexpr int kSelectThreads = 1024, kPer = 8;  // scores that a thread has in flight
constexpr int kMoveThreads = 256, kUnroll = 8, kMoveRows = 256;  // a chunk: up to 2048 vectors of up to 256 rows

struct Select {
    const int32_t *kv_lens;
    int32_t max_tokens, out_tokens, width;
    const float *score;
    int64_t score_stride;
    int32_t budget, sinks, recent;
    int32_t *new_lens, *kept;
    int64_t kept_stride;
    float *out_score;
    int64_t out_score_stride;
    int *err;
};

// An unsigned integer of the same order as the score: NaN lowest, -0 and 0 equal.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (!(x == x)) return 0;
    uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Inclusive scan over a warp's lanes.
__device__ __forceinline__ uint32_t warp_scan(uint32_t x)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, x, d);
        if ((threadIdx.x & 31) >= d) x += o;
    }
    return x;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const Select p)
{
    __shared__ uint32_t hist[2048];
    __shared__ uint32_t sums[32];
    __shared__ uint32_t picked[2];
    grid_dep_entry();
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int given = p.kv_lens[r];
    __syncthreads();  // new_lens may be kv_lens
    const int len = min(max(given, 0), p.max_tokens), fit = min(p.budget, p.out_tokens);
    if (tid == 0 && (given != len || fit < min(len, p.budget))) set_error(p.err, KV_DERR_TABLE);
    const int total = min(len, p.budget);
    const float *scores = p.score + (int64_t)r * p.score_stride;
    const auto score = [&](int j) { return j < p.width ? scores[j] : 0.0f; };  // newer tokens than the scores know weigh nothing yet
    int32_t *kept = p.kept + (int64_t)r * p.kept_stride;
    float *out = p.out_score ? p.out_score + (int64_t)r * p.out_score_stride : nullptr;
    if (tid == 0) p.new_lens[r] = total;
    if (len <= p.budget) {
        for (int i = tid; i < p.budget; i += kSelectThreads) {
            const float s = i < len ? score(i) : 0.0f;
            kept[i] = i < len ? i : -1;
            if (out) out[i] = s;
        }
        return;
    }
    const int a = p.sinks, z = len - p.recent;  // the tokens that compete
    uint32_t want = (uint32_t)(p.budget - p.sinks - p.recent);
    // the key of the last token that stays, eleven (then ten) bits at a time; with none wanted, above all
    uint32_t prefix = 0, mask = 0;
    if (want > 0) {
#pragma unroll
        for (int pass = 0; pass < 3; pass++) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
            const uint32_t zero_bin = (0x80000000u >> shift) & (bins - 1);
            for (int i = tid; i < bins; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
            for (int j0 = a; j0 < z; j0 += kSelectThreads * kPer) {
                float s[kPer];
#pragma unroll
                for (int i = 0; i < kPer; i++) {
                    const int j = j0 + i * kSelectThreads + tid;
                    s[i] = j < z ? score(j) : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < kPer; i++) {
                    if (j0 + i * kSelectThreads >= z) break;
                    uint32_t bin = 0xffffffffu;
                    if (j0 + i * kSelectThreads + tid < z) {
                        const uint32_t k = order_key(s[i]);
                        if ((k & mask) == prefix) bin = (k >> shift) & (bins - 1);
                    }
                    // zeros (most weights of a long request) are added once a warp: their additions to one word
                    // would go one by one
                    const uint32_t zeros = __ballot_sync(0xffffffffu, bin == zero_bin);
                    if (bin == zero_bin) {
                        if (lane == __ffs(zeros) - 1) atomicAdd(&hist[bin], __popc(zeros));
                    } else if (bin != 0xffffffffu) {
                        atomicAdd(&hist[bin], 1);
                    }
                }
            }
            __syncthreads();
            // counts from the top: thread t owns the t-th pair (or single) of bins from the top
            const int each = bins / kSelectThreads;
            uint32_t c[2] = {0, 0}, mine = 0;
            for (int i = 0; i < each; i++) mine += c[i] = hist[bins - 1 - (tid * each + i)];
            const uint32_t upto = warp_scan(mine);
            if (lane == 31) sums[warp] = upto;
            __syncthreads();
            const uint32_t warps = warp_scan(sums[lane]), earlier = __shfl_sync(0xffffffffu, warps, (warp - 1) & 31);
            uint32_t before = upto - mine + (warp ? earlier : 0);
            for (int i = 0; i < each; i++) {
                if (before < want && before + c[i] >= want) {
                    picked[0] = (uint32_t)(bins - 1 - (tid * each + i));
                    picked[1] = want - before;
                }
                before += c[i];
            }
            __syncthreads();
            prefix |= picked[0] << shift;
            mask |= (uint32_t)(bins - 1) << shift;
            want = picked[1];  // of the tokens in this bin
            __syncthreads();
        }
    }
    // the list, in index order: above the key all stay, of the equal ones the first `want`
    const bool some = p.budget > p.sinks + p.recent;
    uint32_t sure0 = 0, ties0 = 0;
    for (int j0 = 0; j0 < len; j0 += kSelectThreads * kPer) {
        float s[kPer];
        uint32_t flags = 0, mine = 0;  // two bits a token; counts: sure in the low half, equal in the high
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const int j = j0 + tid * kPer + i;
            s[i] = j < len ? score(j) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const int j = j0 + tid * kPer + i;
            if (j < len) {
                const uint32_t k = order_key(s[i]);
                if (j < a || j >= z || (some && k > prefix)) {
                    flags |= 1u << (2 * i);
                    mine += 1;
                } else if (some && k == prefix) {
                    flags |= 2u << (2 * i);
                    mine += 1u << 16;
                }
            }
        }
        const uint32_t upto = warp_scan(mine);
        if (lane == 31) sums[warp] = upto;
        __syncthreads();  // also: every score of these tokens has been read before any is written
        const uint32_t warps = warp_scan(sums[lane]), all = __shfl_sync(0xffffffffu, warps, 31);
        const uint32_t earlier = __shfl_sync(0xffffffffu, warps, (warp - 1) & 31), at0 = upto - mine + (warp ? earlier : 0);
        uint32_t sure = sure0 + (at0 & 0xffff), ties = ties0 + (at0 >> 16);
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const uint32_t f = (flags >> (2 * i)) & 3;
            if (f == 1 || (f == 2 && ties < want)) {
                const uint32_t at = sure + min(ties, want);
                kept[at] = j0 + tid * kPer + i;
                if (out) out[at] = s[i];
            }
            sure += f & 1;
            ties += f >> 1;
        }
        sure0 += all & 0xffff;
        ties0 += all >> 16;
        __syncthreads();
    }
}

struct Move {
    uint64_t base[kMaxTensorsPerLaunch];
    int32_t n_planes, slices;       // column slices of a row
    FastDiv per;                    // 16-byte vectors of a slice
    int32_t row_vecs;               // of a row
    int32_t num_blocks;
    FastDiv block;
    int64_t block_stride, plane_stride, token_stride;
    const int32_t *table, *out_table;
    int64_t table_stride, out_stride;
    const int32_t *new_lens, *kept;
    int64_t kept_stride;
    int32_t out_tokens, row_parts;
    int *err;
};

// grid: (tensor, plane, slice) x (request, stretch of its list)
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ Move p)
{
    constexpr int kVecs = kMoveThreads * kUnroll;
    __shared__ int64_t from[2][kMoveRows], to[2][kMoveRows];
    grid_dep_entry();
    const int tid = threadIdx.x;
    const int slice = blockIdx.x % p.slices, tp = blockIdx.x / p.slices, plane = tp % p.n_planes, tensor = tp / p.n_planes;
    const int r = blockIdx.y / p.row_parts, part = blockIdx.y % p.row_parts;
    const int n = min(__ldg(p.new_lens + r), p.out_tokens);
    const int i0 = (int)((int64_t)n * part / p.row_parts), i1 = (int)((int64_t)n * (part + 1) / p.row_parts);
    char *base = (char *)p.base[tensor] + plane * p.plane_stride + (int64_t)slice * p.per.d * 16;
    const int vecs = min((int)p.per.d, p.row_vecs - slice * (int)p.per.d);
    const int rows = min(kMoveRows, kVecs / (int)p.per.d);
    const int32_t *kept = p.kept + (int64_t)r * p.kept_stride;
    const int32_t *row = p.table + (int64_t)r * p.table_stride, *out_row = p.out_table + (int64_t)r * p.out_stride;
    const auto offset = [&](const int32_t *t, int j) {
        const uint32_t col = fdiv((uint32_t)j, p.block);
        const int page = __ldg(t + col);
        if (page < 0 || page >= p.num_blocks) {
            set_error(p.err, KV_DERR_TABLE);
            return (int64_t)-1;
        }
        return page * p.block_stride + (j - (int64_t)(col * p.block.d)) * p.token_stride;
    };
    const auto look = [&](int i, int k) {  // the offsets of a chunk's rows; -1: nothing to move
        for (int x = tid; x < rows; x += kMoveThreads) {
            int64_t f = -1, t = -1;
            if (i + x < i1) {
                f = offset(row, __ldg(kept + i + x));
                t = offset(out_row, i + x);
                if (f == t || t < 0) f = -1;
            }
            from[k][x] = f;
            to[k][x] = t;
        }
    };
    look(i0, 0);
    __syncthreads();
    int k = 0;
    for (int i = i0; i < i1; i += rows, k ^= 1) {
        uint4 v[kUnroll];
        int64_t at[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const uint32_t e = (uint32_t)(u * kMoveThreads + tid), x = fdiv(e, p.per), c = e - x * p.per.d;
            at[u] = -1;
            if ((int)x < rows && (int)c < vecs) {
                const int64_t f = from[k][x];
                if (f >= 0) {
                    v[u] = *reinterpret_cast<const uint4 *>(base + f + c * 16);
                    at[u] = to[k][x] + c * 16;
                }
            }
        }
        look(i + rows, k ^ 1);
        __syncthreads();  // all loads of the chunk stand before its stores
#pragma unroll
        for (int u = 0; u < kUnroll; u++)
            if (at[u] >= 0) st_stream(base + at[u], v[u]);
    }
}

}  // namespace

int preload_evict_kernels() { return load_kernels(evict_select_kernel, evict_move_kernel); }

}  // namespace pkv

using namespace pkv;

extern "C" int kv_evict(const kv_cache_desc *cache, const int32_t *block_table, int32_t n_reqs, int32_t max_blocks_per_req,
                        int64_t bt_row_stride, const int32_t *kv_lens, const float *score, int64_t score_stride, int32_t width, int32_t budget,
                        int32_t sinks, int32_t recent, const int32_t *out_table, int32_t out_blocks_per_req, int64_t out_row_stride,
                        int32_t *new_lens, int32_t *kept, int64_t kept_stride, float *out_score, int64_t out_score_stride, kv_stream_t stream)
{
    int st = check_cache(cache);
    if (st != KV_OK) return st;
    if (n_reqs < 0 || max_blocks_per_req < 0 || out_blocks_per_req < 0 || bt_row_stride < 0 || out_row_stride < 0 || width < 0 || budget < 0 ||
        sinks < 0 || recent < 0 || score_stride < 0 || kept_stride < 0 || out_score_stride < 0)
        return KV_ERR_INVALID_ARG;
    if ((int64_t)sinks + recent > budget) return KV_ERR_INVALID_ARG;
    if (n_reqs == 0) return KV_OK;
    if (kv_lens == nullptr || new_lens == nullptr || (kept == nullptr && budget > 0) || (score == nullptr && width > 0) ||
        (block_table == nullptr && max_blocks_per_req > 0) || (out_table == nullptr && out_blocks_per_req > 0))
        return KV_ERR_INVALID_ARG;
    if (n_reqs > 1 && (bt_row_stride < max_blocks_per_req || out_row_stride < out_blocks_per_req || score_stride < width || kept_stride < budget ||
                       (out_score != nullptr && out_score_stride < budget)))
        return KV_ERR_INVALID_ARG;
    if (((uintptr_t)score & 3u) || ((uintptr_t)out_score & 3u)) return KV_ERR_ALIGN;
    const int64_t max_tokens = (int64_t)max_blocks_per_req * cache->block_size, out_tokens = (int64_t)out_blocks_per_req * cache->block_size;
    if (max_tokens > (1ll << 30) || out_tokens > (1ll << 30) || cache->num_blocks >= (1ll << 31) || n_reqs > 65535 || budget > (1 << 30))
        return KV_ERR_UNSUPPORTED;
    const DeviceInfo *dev = current_device();
    if (dev == nullptr) return KV_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    const Select sel{kv_lens, (int32_t)max_tokens, (int32_t)out_tokens, width, score, score_stride, budget, sinks, recent, new_lens, kept,
                     kept_stride, out_score, out_score_stride, dev->err_word};
    if ((st = cuda_status(launch(evict_select_kernel, dim3(n_reqs), dim3(kSelectThreads), 0, s, sel))) != KV_OK) return st;
    if (cache->n_tensors == 0 || out_tokens == 0 || budget == 0) return KV_OK;
    Move m = {};
    m.n_planes = cache->n_planes;
    m.row_vecs = cache->row_bytes / 16;
    m.slices = (m.row_vecs + 511) / 512;
    m.per = make_fastdiv((uint32_t)((m.row_vecs + m.slices - 1) / m.slices));
    m.num_blocks = (int32_t)cache->num_blocks;
    m.block = make_fastdiv((uint32_t)cache->block_size);
    m.block_stride = cache->block_stride;
    m.plane_stride = cache->n_planes == 2 ? cache->plane_stride : 0;
    m.token_stride = cache->token_stride;
    m.table = block_table;
    m.out_table = out_table;
    m.table_stride = bt_row_stride;
    m.out_stride = out_row_stride;
    m.new_lens = new_lens;
    m.kept = kept;
    m.kept_stride = kept_stride;
    m.out_tokens = (int32_t)out_tokens;
    m.err = dev->err_word;
    for (int t0 = 0; t0 < cache->n_tensors; t0 += kMaxTensorsPerLaunch) {
        const int nt = cache->n_tensors - t0 < kMaxTensorsPerLaunch ? cache->n_tensors - t0 : kMaxTensorsPerLaunch;
        for (int i = 0; i < nt; i++) m.base[i] = cache->base[t0 + i];
        const int columns = nt * m.n_planes * m.slices;
        // in place one CTA walks a whole list; into other pages its stretches may go side by side
        m.row_parts = 1;
        if (out_table != block_table) {
            const int64_t rows = std::min<int64_t>(kMoveRows, kMoveThreads * kUnroll / m.per.d), chunks = (budget + rows - 1) / rows;
            int64_t want = ((int64_t)dev->num_sms * 8 + (int64_t)columns * n_reqs - 1) / ((int64_t)columns * n_reqs);
            if (want > chunks) want = chunks;
            if (want > 65535 / n_reqs) want = 65535 / n_reqs;
            if (want > 1) m.row_parts = (int32_t)want;
        }
        if ((st = cuda_status(launch<false>(evict_move_kernel, dim3(columns, n_reqs * m.row_parts), dim3(kMoveThreads), 0, s, m))) != KV_OK) return st;
    }
    return KV_OK;
}
