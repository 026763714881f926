// kv_attention_mass: the attention weight that every cached token receives.
//
//   score[r, j] = prev[r, j] + sum over the request's new tokens t that see j, and over the query heads h,
//                 of exp(scale q[t, h] . K[j] - lse[t, h])
//
// The products are formed with keys as the rows of the accumulator, S^T = K Q^T: a thread owns a key and adds
// the exponentials of its row, column by column in a fixed order, so nothing is shared and nothing atomic.
// The line (as in kv_plan.cuh) runs over requests, tiles of 128 keys, key heads and tiles of up to 128
// (token, head of the group) rows; a CTA takes an equal piece of it, and a key tile that was cut is summed
// from its pieces' partial sums, in their order, by whichever CTA finishes the last of them.
//   warps 0 and 2 load K once a head, warp 3 Q and warps 12 and 13 its rows' normalisers a step, warp 1
//   issues the products into four accumulators (all of tensor memory: the exponentials take longer than
//   the products), warps 4-7 and 8-11 take the even and the odd steps.  Warp 2 ends with what lies past
//   the requests' lengths.
// A decode step is bound by memory once there is enough of it: 128 requests of 6000 to 8000 tokens, 32 heads over 8,
// take 293 us, 93% of the copy rate (16 of 2000 to 6000: 32 us, 65%).  Chunks are bound by a step's 512 cycles of
// exponentials and 768 of shared memory (operands and the normalisers that every thread reads): four of 512 to 1024
// tokens over 4000 to 8000 take 134 us.
#include "kv_attention.cuh"

namespace pkv {

namespace {

constexpr int kLeast = 2;  // steps of a piece of a unit, at least
constexpr int kThreads = 448;
constexpr int kTileShift = 7, kTile = 1 << kTileShift;
constexpr uint32_t kPanel = 128 * 128, kAuxBytes = 3 << 10;

template <int DK>
struct Shape {
    static constexpr uint32_t kOperand = 128 * DK * 2;
    static constexpr int kNK = DK == 64 ? 8 : DK == 128 ? 4 : 2, kNQ = DK == 64 ? 4 : DK == 128 ? 3 : 2;  // what 227 KB holds
    static constexpr uint32_t kOffQ = kNK * kOperand, kOffAux = kOffQ + kNQ * kOperand, kBytes = kOffAux + kAuxBytes;
};

struct Params {
    Batch b;
    const int32_t *table;
    int64_t table_stride;
    int32_t num_blocks;
    FastDiv block;
    int32_t piece_rows, dk, heads;
    int32_t step_tokens;  // tokens of one step: 128 / group
    FastDiv step;
    int32_t q_box;        // tokens one TMA brings of q, a divisor of step_tokens
    float c;
    const float *lse;
    const float *prev;
    int64_t prev_stride;
    float *score;
    int64_t score_stride;
    int32_t width;
    float *ws;
    int *counters;
};

struct Aux {
    uint64_t k_full[8], k_empty[8], q_full[4], q_empty[4], s_full[4], s_empty[4], l_full[4], sum_ready, sum_free, join;
    Place place;
    alignas(16) float neg[4][128];  // read four at a time: -lse log2 e of a step's rows
    float odd[128];     // the odd steps' sums
    uint32_t tmem;
    int answer;
    int gave_up;
};
static_assert(sizeof(Aux) <= kAuxBytes, "bookkeeping");

// The steps of one key tile: a key head's query rows, in steps of step_tokens tokens.
struct KeyTile {
    int t0, t1;     // tokens that see some key of the tile
    int per_head;   // steps of a key head
    int steps;      // of the tile (at least one: its scores have to be written)
    int lo;         // first key that some token sees
};

__device__ __forceinline__ KeyTile key_tile(const Params &p, const Request &q, int tile)
{
    const Batch &b = p.b;
    const int kb = tile * kTile, end = min(kb + kTile, q.len), base = q.len - q.q_len;
    KeyTile k;
    k.t0 = b.causal ? max(0, kb - base) : 0;
    k.t1 = b.window ? min(q.q_len, max(0, end - 1 + b.window - base)) : q.q_len;
    k.per_head = k.t1 > k.t0 ? (int)fdiv((uint32_t)(k.t1 - k.t0 + p.step_tokens - 1), p.step) : 0;
    k.steps = max(1, k.per_head * b.kv_heads);
    k.lo = b.window ? max(0, base - b.window + 1) : 0;
    return k;
}

// The request's first key tiles that all take the same number of steps: without a window those that every
// new token sees from their first key on, with one those that no token sees.
__device__ __forceinline__ int even_tiles(const Params &p, const Request &q)
{
    const Batch &b = p.b;
    const int tiles = (q.len + kTile - 1) / kTile, base = q.len - q.q_len;
    if (b.window) return min(tiles, max(0, base - b.window + 1) / kTile);
    if (!b.causal) return tiles;
    return base < 0 ? 0 : min(tiles, base / kTile + 1);
}

// The line: a unit is a key tile.
struct MassWork {
    static constexpr int kSnap = 0;
    const Params &p;
    bool report;
    // sum over the request's key tiles of their pieces of `each` steps
    __device__ __forceinline__ int count(const Request &q, int each) const
    {
        int t = even_tiles(p, q), n = t > 0 ? t * ceil_div(key_tile(p, q, 0).steps, each) : 0;
#pragma unroll 1
        for (; t * kTile < q.len; t++) n += ceil_div(key_tile(p, q, t).steps, each);
        return n;
    }
    __device__ __forceinline__ void measure(int r, int &steps, int &units) const
    {
        const Request q = load_request(p.b, r, report);
        steps = add_steps(steps, count(q, 1));
        units += (q.len + kTile - 1) / kTile;
    }
    __device__ __forceinline__ int pieces(int r, int each) const { return count(load_request(p.b, r), each); }
    __device__ __forceinline__ Place own(int r, int k, int each) const
    {
        const Request q = load_request(p.b, r);
        Place pl;
        pl.req = r, pl.head = 0, pl.unit = 0;
        const int even = even_tiles(p, q);
        if (even > 0) {
            const int n = ceil_div(key_tile(p, q, 0).steps, each);
            pl.unit = min(even, (int)((uint32_t)k / (uint32_t)n));
            k -= pl.unit * n;
        }
        int steps = 0;
#pragma unroll 1
        for (;; pl.unit++) {
            steps = key_tile(p, q, pl.unit).steps;
            const int n = ceil_div(steps, each);
            if (k < n) break;
            k -= n;
        }
        pl.nth = k;
        pl.off = k * each;
        pl.steps = min(each, steps - pl.off);
        return pl;
    }
};

// Walks a piece key tile by key tile.  place.unit: the key tile; place.off: the step inside it.
struct Walk2 {
    Place at;
    int left, n;
    int pos;  // the fragment's first step on the line
    Request q;
    KeyTile k;
    __device__ __forceinline__ bool start(const Params &p, const Place &pl, const Line &line)
    {
        at = pl;
        left = line.steps;
        pos = line.begin;
        if (left <= 0) return false;
        q = load_request(p.b, at.req);
        k = key_tile(p, q, at.unit);
        n = min(left, k.steps - at.off);
        return true;
    }
    __device__ __forceinline__ bool next(const Params &p)
    {
        left -= n;
        pos += n;
        if (left <= 0) return false;
        at.off = 0;
        at.unit++;
        while (at.unit * kTile >= q.len) {
            at.unit = 0;
            q = load_request(p.b, ++at.req);
        }
        k = key_tile(p, q, at.unit);
        n = min(left, k.steps);
        return true;
    }
};

template <int DK, bool Bf16>
__global__ void __launch_bounds__(kThreads, 1)
mass_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap q_map, const Params p)
{
    using S = Shape<DK>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    Aux &aux = *reinterpret_cast<Aux *>(smem + S::kOffAux);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const Batch &b = p.b;
    const Waiter wait{&aux.gave_up, b.err};
    const int group = (int)b.group.d;

    if (tid == 0) {
        aux.gave_up = 0;
        for (int i = 0; i < S::kNK; i++) mbar_init(smem_addr(&aux.k_full[i]), 2), mbar_init(smem_addr(&aux.k_empty[i]), 1);
        for (int i = 0; i < S::kNQ; i++) mbar_init(smem_addr(&aux.q_full[i]), 1), mbar_init(smem_addr(&aux.q_empty[i]), 1);
        for (int i = 0; i < 4; i++) {
            mbar_init(smem_addr(&aux.s_full[i]), 1);
            mbar_init(smem_addr(&aux.s_empty[i]), 4);
            mbar_init(smem_addr(&aux.l_full[i]), 1);
        }
        mbar_init(smem_addr(&aux.sum_ready), 4);
        mbar_init(smem_addr(&aux.sum_free), 4);
        mbar_init(smem_addr(&aux.join), 4);
        mbar_init_fence();
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&q_map);
    }
    if (warp == 2) tmem_alloc(smem_addr(&aux.tmem), 512);
    grid_dep_entry();
    const Line line = find_piece<kThreads>(b.n_reqs, blockIdx.x, gridDim.x, kLeast, reinterpret_cast<int *>(aux.neg), &aux.place, MassWork{p, blockIdx.x == 0});
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, aux.tmem, 0);
    Walk2 w;
    if (!w.start(p, aux.place, line)) {
        // nothing to do: on to the common exit
    } else if (warp == 0 || warp == 2) {
        // ---- keys: the two warps take every other page piece (one warp issues a TMA in about 140 cycles, which
        // for pages of 16 slots held the whole kernel to 60% of the memory's rate) ----
        const int pr = p.piece_rows, mine = warp >> 1;
        int kt = 0;
        bool ok = true;
        do {
            if (w.k.per_head == 0) continue;
            const int kb = w.at.unit * kTile, p0 = max(0, w.k.lo - kb) / pr, p1 = (min(w.q.len - kb, kTile) + pr - 1) / pr;
            const int32_t *row = p.table + (int64_t)w.at.req * p.table_stride;
            int page = 0, slot = 0;
            const auto find = [&](int j) {
                const uint32_t key = (uint32_t)(kb + j * pr), col = fdiv(key, p.block);
                slot = (int)(key - col * p.block.d);
                page = __ldg(row + col);
                if (page < 0 || page >= p.num_blocks) {
                    set_error(b.err, KV_DERR_TABLE);
                    page = p.num_blocks;  // outside the map: reads zeros
                }
            };
            const int first = p0 + mine + 2 * lane, count = (p1 - p0 - mine + 1) / 2;
            if (first < p1) find(first);  // this lane's first page, the same for every head
            const int page0 = page, slot0 = slot;
            const int head0 = w.at.off / w.k.per_head, head1 = (w.at.off + w.n - 1) / w.k.per_head;
            for (int head = head0; head <= head1; head++, kt++) {
                const int s = kt % S::kNK;
                const uint32_t bar = smem_addr(&aux.k_full[s]);
                if (kt >= S::kNK && !wait.warp(smem_addr(&aux.k_empty[s]), ((kt / S::kNK) - 1) & 1)) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(count * pr) * DK * 2);
                __syncwarp();
                page = page0, slot = slot0;
                for (int j = first; j < p1; j += 64) {
                    if (j >= p0 + 64) find(j);
#pragma unroll
                    for (int h = 0; h < DK / 64; h++)
                        tma_load_4d(base + s * S::kOperand + h * kPanel + j * pr * 128, &k_map, bar, h * 64, head, slot, page);
                }
                __syncwarp();
            }
        } while (ok && w.next(p));
    } else if (warp == 3) {
        // ---- queries ----
        int it = 0;
        bool ok = true;
        do {
            if (w.k.per_head == 0) continue;
            const int tok_first = w.q.q0 + w.k.t0, ntok = w.k.t1 - w.k.t0;
            int head = w.at.off / w.k.per_head, qi = w.at.off - head * w.k.per_head;
            for (int i = 0; i < w.n; i++, it++) {
                const int tok0 = qi * p.step_tokens, toks = min(p.step_tokens, ntok - tok0), s = it % S::kNQ;
                if (it >= S::kNQ && !(ok = wait.warp(smem_addr(&aux.q_empty[s]), ((it / S::kNQ) - 1) & 1))) break;
                const uint32_t bar = smem_addr(&aux.q_full[s]);
                const int boxes = (toks + p.q_box - 1) / p.q_box;
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * p.q_box * group) * DK * 2);
                __syncwarp();
                for (int j = lane; j < boxes; j += 32)
#pragma unroll
                    for (int h = 0; h < DK / 64; h++)
                        tma_load_3d(base + S::kOffQ + s * S::kOperand + h * kPanel + j * p.q_box * group * 128, &q_map, bar, h * 64, head * group,
                                    tok_first + tok0 + j * p.q_box);
                __syncwarp();
                if (++qi == w.k.per_head) qi = 0, head++;
            }
        } while (ok && w.next(p));
    } else if (warp >= 12) {
        // ---- the normalisers of a step's rows, a warp for the even steps and one for the odd: a trip to memory
        // takes longer than a step ----
        int it = 0;
        bool ok = true;
        do {
            if (w.k.per_head == 0) continue;
            const int tok_first = w.q.q0 + w.k.t0, ntok = w.k.t1 - w.k.t0;
            int head = w.at.off / w.k.per_head, qi = w.at.off - head * w.k.per_head;
            for (int i = 0; i < w.n; i++, it++) {
                if ((it & 1) == warp - 12) {
                    const int tok0 = qi * p.step_tokens, cols = min(p.step_tokens, ntok - tok0) * group, s = it & 3;
                    float v[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int c = j * 32 + lane, tt = (int)fdiv((uint32_t)c, b.group);
                        v[j] = c < cols ? -p.lse[(int64_t)(tok_first + tok0 + tt) * p.heads + head * group + c - tt * group] * kLog2e : -INFINITY;
                        if (v[j] == INFINITY) v[j] = -INFINITY;  // a row that saw nothing weighs nothing
                    }
                    if (it >= 4 && !(ok = wait.warp(smem_addr(&aux.s_empty[s]), ((it >> 2) - 1) & 1))) break;
#pragma unroll
                    for (int j = 0; j < 4; j++) aux.neg[s][j * 32 + lane] = v[j];
                    warp_arrive(smem_addr(&aux.l_full[s]));
                }
                if (++qi == w.k.per_head) qi = 0, head++;
            }
        } while (ok && w.next(p));
    } else if (warp == 1) {
        const uint32_t elected = elect_one();
        const uint64_t kd = smem_desc(base, 16, 1024), qd = smem_desc(base + S::kOffQ, 16, 1024);
        int kt = -1, it = 0;
        bool ok = true;
        do {
            if (w.k.per_head == 0) continue;
            int qi = w.at.off % w.k.per_head;
            for (int i = 0; ok && i < w.n; i++, it++) {
                const int s = it % S::kNQ;
                const int rows = min(p.step_tokens, w.k.t1 - w.k.t0 - qi * p.step_tokens) * group;
                const uint32_t desc = mma_desc(Bf16, 128, (uint32_t)(rows + 15) & ~15u, false);
                if (i == 0 || qi == 0) kt++;  // another head's K
                const uint32_t k_bar = smem_addr(&aux.k_full[kt % S::kNK]), q_bar = smem_addr(&aux.q_full[s]);
                const uint32_t k_parity = (kt / S::kNK) & 1, q_parity = (it / S::kNQ) & 1;
                ok = it < 4 ? wait.warp(k_bar, k_parity, q_bar, q_parity)
                            : wait.warp(k_bar, k_parity, q_bar, q_parity, smem_addr(&aux.s_empty[it & 3]), ((it >> 2) - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t ka = kd + (kt % S::kNK) * (S::kOperand >> 4), qa = qd + s * (S::kOperand >> 4);
#pragma unroll
                for (int kk = 0; kk < DK / 16; kk++) {
                    const uint32_t o = ((kk / 4) * kPanel + (kk % 4) * 32) >> 4;
                    mma_ss(tmem + (it & 3) * 128, ka + o, qa + o, desc, kk > 0, elected);
                }
                tc_commit(smem_addr(&aux.q_empty[s]), elected);
                if (++qi == w.k.per_head) qi = 0;
                if (i + 1 == w.n || qi == 0) tc_commit(smem_addr(&aux.k_empty[kt % S::kNK]), elected);
                tc_commit(smem_addr(&aux.s_full[it & 3]), elected);  // last: the groups wait for it before the CTA ends
            }
        } while (ok && w.next(p));
    } else if (warp >= 4) {
        const int g = (warp - 4) >> 2, t = tid & 127;
        const uint32_t mine = (uint32_t)((warp & 3) * 32) << 16;
        int it = 0, tiles = 0, cuts = 0;
        bool ok = true;
        do {
            const int key = w.at.unit * kTile + t;
            float sum = 0.0f;
            if (w.k.per_head) {
                const int ntok = w.k.t1 - w.k.t0, base_pos = w.q.len - w.q.q_len + w.k.t0;
                // tokens (counted from t0) that see this key: [va, vb)
                const int va = b.causal ? max(0, key - base_pos) : 0, vb = key >= w.q.len ? 0 : b.window ? min(ntok, max(0, key + b.window - base_pos)) : ntok;
                int qi = w.at.off % w.k.per_head - 1;
                for (int i = 0; i < w.n; i++, it++) {
                    if (++qi == w.k.per_head) qi = 0;
                    if ((it & 1) != g) continue;
                    const int tok0 = qi * p.step_tokens;
                    const uint32_t s_at = tmem + (it & 3) * 128 + mine;
                    const int cols = min(p.step_tokens, ntok - tok0) * group;
                    if (!wait.warp(smem_addr(&aux.l_full[it & 3]), (it >> 2) & 1) || !wait.warp(smem_addr(&aux.s_full[it & 3]), (it >> 2) & 1)) { ok = false; break; }
                    tc_fence_after();
                    const int c0 = (va - tok0) * group, c1 = min(cols, (vb - tok0) * group);
                    float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    const auto add = [&](const uint32_t(&x)[32], int q) {
                        const float4 *neg = reinterpret_cast<const float4 *>(&aux.neg[it & 3][q]);
                        const float2 cc = make_float2(p.c, p.c);
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const float4 n = neg[j];
                            float2 e = fma2(make_float2(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1])), cc, make_float2(n.x, n.y));
                            float2 f = fma2(make_float2(__uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3])), cc, make_float2(n.z, n.w));
                            e.x = exp2_fast(e.x), e.y = exp2_fast(e.y), f.x = exp2_fast(f.x), f.y = exp2_fast(f.y);
                            part[0] = add2(part[0], e);
                            part[1] = add2(part[1], f);
                        }
                    };
                    uint32_t x0[32], x1[32];
                    if (__any_sync(0xffffffffu, c0 > 0 || c1 < 128)) {  // some key is not seen by some row, or rows are missing
#pragma unroll 1
                        for (int q = 0; q < cols; q += 32) {
                            tmem_ld32(s_at + q, x0);
                            tc_wait_ld();
                            hide32(x0, c0 - q, c1 - q);
                            add(x0, q);
                        }
                    } else {  // 32 columns are read while 32 are added
                        tmem_ld32(s_at, x0);
                        tc_wait_ld();
                        tmem_ld32(s_at + 32, x1);
                        add(x0, 0);
                        tc_wait_ld();
                        tmem_ld32(s_at + 64, x0);
                        add(x1, 32);
                        tc_wait_ld();
                        tmem_ld32(s_at + 96, x1);
                        add(x0, 64);
                        tc_wait_ld();
                        add(x1, 96);
                    }
                    sum += (part[0].x + part[0].y) + (part[1].x + part[1].y);
                    tc_fence_before();
                    warp_arrive(smem_addr(&aux.s_empty[it & 3]));
                }
                if (!ok) break;
            }
            // the odd steps' group hands its sums over
            if (g == 1) {
                if (tiles && !wait.warp(smem_addr(&aux.sum_free), (tiles - 1) & 1)) { ok = false; break; }
                aux.odd[t] = sum;
                warp_arrive(smem_addr(&aux.sum_ready));
            } else {
                if (!wait.warp(smem_addr(&aux.sum_ready), tiles & 1)) { ok = false; break; }
                sum += aux.odd[t];
                warp_arrive(smem_addr(&aux.sum_free));
                bool mine_to_write = true;
                if (w.n < w.k.steps) {  // cut: the group that comes last adds the fragments in their order
                    const Cut cut(line, w.pos - w.at.off, w.k.steps);
                    p.ws[(2 * blockIdx.x + (w.at.off == 0 ? 1 : 0)) * kTile + t] = sum;
                    mine_to_write = last_of(p.counters + cut.c0, cut.count, smem_addr(&aux.join), cuts, &aux.answer, wait, ok);
                    if (!ok) break;
                    if (mine_to_write) {
                        sum = 0.0f;
#pragma unroll 4
                        for (int i = 0; i < cut.count; i++) sum += __ldcg(p.ws + cut.slot(i) * kTile + t);
                    }
                }
                if (mine_to_write && key < w.q.len && key < p.width)
                    p.score[(int64_t)w.at.req * p.score_stride + key] = sum + (p.prev ? p.prev[(int64_t)w.at.req * p.prev_stride + key] : 0.0f);
            }
            tiles++;
        } while (w.next(p));
        (void)ok;
    }
    if (warp == 2) {
        // what lies past every request's length is carried over, a piece of up to 1024 columns at a time
        const int each = (p.width + 1023) >> 10;
#pragma unroll 1
        for (int i = blockIdx.x; i < b.n_reqs * each; i += gridDim.x) {
            const int r = i / each, j0 = (i - r * each) << 10, len = min(max(__ldg(b.kv_lens + r), 0), b.max_tokens);
            const int end = min(j0 + 1024, p.width);
            for (int j = max(j0, len) + lane; j < end; j += 256) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; k++) v[k] = p.prev && j + 32 * k < end ? p.prev[(int64_t)r * p.prev_stride + j + 32 * k] : 0.0f;
#pragma unroll
                for (int k = 0; k < 8; k++)
                    if (j + 32 * k < end) p.score[(int64_t)r * p.score_stride + j + 32 * k] = v[k];
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
    if (warp == 2) tmem_free(tmem, 512);
}

template <int DK, bool Bf16>
int run_mass(const CUtensorMap &km, const CUtensorMap &qm, const Params &p, int parts, cudaStream_t s, bool prepare)
{
    if (prepare)
        return cuda_status(cudaFuncSetAttribute(mass_kernel<DK, Bf16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<DK>::kBytes));
    return cuda_status(launch(mass_kernel<DK, Bf16>, dim3(parts), dim3(kThreads), Shape<DK>::kBytes, s, km, qm, p));
}

template <bool Bf16>
int pick_mass(int dk, const CUtensorMap &km, const CUtensorMap &qm, const Params &p, int parts, cudaStream_t s, bool prepare)
{
    if (dk <= 64) return run_mass<64, Bf16>(km, qm, p, parts, s, prepare);
    if (dk <= 128) return run_mass<128, Bf16>(km, qm, p, parts, s, prepare);
    return run_mass<192, Bf16>(km, qm, p, parts, s, prepare);
}

int64_t mass_workspace(int num_sms) { return kCounterBytes + (int64_t)num_sms * 2 * kTile * 4; }

}  // namespace

int preload_mass_kernels()
{
    Params p = {};
    CUtensorMap m;
    for (int dk : {64, 128, 192})
        for (bool bf : {false, true}) {
            const int st = bf ? pick_mass<true>(dk, m, m, p, 0, nullptr, true) : pick_mass<false>(dk, m, m, p, 0, nullptr, true);
            if (st != KV_OK) return st;
        }
    return load_kernels(mass_kernel<64, false>, mass_kernel<64, true>, mass_kernel<128, false>, mass_kernel<128, true>,
                        mass_kernel<192, false>, mass_kernel<192, true>);
}

}  // namespace pkv

using namespace pkv;

extern "C" {

int kv_attention_mass_workspace_bytes(int64_t *bytes_out)
{
    if (bytes_out == nullptr) return KV_ERR_INVALID_ARG;
    const DeviceInfo *d = current_device();
    if (d == nullptr) return KV_ERR_CUDA;
    *bytes_out = mass_workspace(d->num_sms);
    return KV_OK;
}

int kv_attention_mass(const kv_attn_desc *d, const kv_attn_batch *batch, const kv_cache_desc *k, int32_t k_tensor, int32_t k_plane,
                      const void *q, int64_t q_token_stride, int64_t q_head_stride, const float *lse, const float *prev,
                      int64_t prev_stride, float *score, int64_t score_stride, int32_t width, void *workspace, int64_t workspace_bytes,
                      kv_stream_t stream)
{
    if (d == nullptr || d->n_heads <= 0 || d->n_kv_heads <= 0 || d->n_heads % d->n_kv_heads != 0 || d->head_dim <= 0 || d->window < 0 ||
        !good_scale(d->scale) || (d->dtype != KV_BF16 && d->dtype != KV_F16) || width < 0)
        return KV_ERR_INVALID_ARG;
    int st = check_batch(batch);
    if (st != KV_OK) return st;
    if (d->head_dim % 8) return KV_ERR_ALIGN;
    if (d->head_dim > 192 || d->n_heads / d->n_kv_heads > 128 || (d->window && !d->causal) || width > (1 << 30)) return KV_ERR_UNSUPPORTED;
    if ((st = check_plane(k, k_tensor, k_plane, d->n_kv_heads, d->head_dim)) != KV_OK) return st;
    if (batch->n_reqs == 0 || width == 0) return KV_OK;
    if (batch->n_tokens > 0) {
        if ((st = check_rows(q, q_token_stride, q_head_stride)) != KV_OK) return st;
        if (lse == nullptr) return KV_ERR_INVALID_ARG;
    }
    if (score == nullptr || workspace == nullptr || score_stride < 0 || prev_stride < 0) return KV_ERR_INVALID_ARG;
    if (batch->n_reqs > 1 && (score_stride < width || (prev != nullptr && prev_stride < width))) return KV_ERR_INVALID_ARG;
    if (!aligned16(workspace) || ((uintptr_t)lse & 3u) || ((uintptr_t)prev & 3u) || ((uintptr_t)score & 3u)) return KV_ERR_ALIGN;
    const int group = d->n_heads / d->n_kv_heads;
    Params p = {};
    if ((st = fill_batch(&p.b, batch, d->n_heads, d->n_kv_heads, k->block_size, 128 / group * group, kTileShift, d->causal, d->window)) != KV_OK) return st;
    const DeviceInfo *dev = current_device();
    if (dev == nullptr) return KV_ERR_CUDA;
    if (workspace_bytes < mass_workspace(dev->num_sms)) return KV_ERR_RANGE;
    if ((st = prepare_attention(*dev)) != KV_OK) return st;
    p.b.err = dev->err_word;
    p.table = batch->block_table;
    p.table_stride = batch->bt_row_stride;
    p.num_blocks = (int32_t)k->num_blocks;
    p.block = make_fastdiv((uint32_t)k->block_size);
    p.piece_rows = piece_rows(k->block_size, kTile);
    p.dk = d->head_dim;
    p.heads = d->n_heads;
    p.step_tokens = 128 / group;
    p.step = make_fastdiv((uint32_t)p.step_tokens);
    p.q_box = box_tokens(p.step_tokens, batch);
    p.c = d->scale * kLog2e;
    p.lse = lse;
    p.prev = prev;
    p.prev_stride = prev_stride;
    p.score = score;
    p.score_stride = score_stride;
    p.width = width;
    p.counters = (int *)workspace;
    p.ws = (float *)((char *)workspace + kCounterBytes);
    CUtensorMap km, qm;
    if ((st = make_cache_map(&km, k, k_tensor, k_plane, d->n_kv_heads, d->head_dim, p.piece_rows)) != KV_OK) return st;
    if (batch->n_tokens > 0) {
        if ((st = make_q_map(&qm, q, q_token_stride, q_head_stride, d->head_dim, d->n_heads, batch->n_tokens, group, p.q_box)) != KV_OK)
            return st;
    } else {
        qm = km;  // never used: no request has new tokens
    }
    return d->dtype == KV_BF16 ? pick_mass<true>(p.dk, km, qm, p, dev->num_sms, (cudaStream_t)stream, false)
                               : pick_mass<false>(p.dk, km, qm, p, dev->num_sms, (cudaStream_t)stream, false);
}

}  // extern "C"
