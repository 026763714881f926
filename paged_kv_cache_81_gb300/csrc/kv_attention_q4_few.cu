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
// Queries are brought to [1, 2) by a power of two a row and held in fp16, weights are fp16 (kv_tensor.cuh, weight_offset);
// sums are in 32 bits.
//
// One persistent CTA per SM; a unit is one request's rows of up to eight key heads.
//   warp 0        brings rows of keys and of values by tiled TMA, one for each run of slots inside a page, into rings of tiles
//   other warps   each one key head and every n-th 16 keys of a tile: scores, weights, values, with a running maximum and sum of
//                 its own, joined through shared memory at the unit's end
// Rows lie 32 or 96 bytes off a multiple of 128 apart and the 16 keys of a step are taken in an order (kOrder) in which neither the
// keys' 16-byte nor the values' 8-byte reads meet in a bank.
#include "kv_attention_q4.cuh"

namespace pkv {

namespace {

constexpr int kLeast = 2;     // tiles of a piece of a unit, at least
constexpr int kMaxHeads = 8;  // key heads of a unit
constexpr int kMaxSlots = 4;
constexpr uint32_t kOrder = 0x57463120u;  // key of row r of 8: hexadecimal digit r

template <int D, int NT>
struct Few {
    static constexpr int kWarps = NT == 1 ? 16 : 8;  // that compute
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int kRows = 8 * NT;
    static constexpr int kSteps = NT == 1 ? 2 : 4;   // groups of 16 keys that a warp takes of a tile
    static constexpr int kPitch = D + 4;             // floats of a row in the join
    static constexpr uint32_t kJoin = (uint32_t)kWarps * kRows * kPitch * 4;
    // bytes between a tile's rows of H heads of D, 32 off a multiple of 64
    static constexpr uint32_t pitch(int h) { return (uint32_t)((h * D * 9 + 255) / 256 * 16 - 32 + 63) / 64 * 64 + 32; }
};
static_assert(kMaxHeads * Few<128, 2>::kRows <= 256, "a fragment fits its place in the workspace");

// Where a unit's heads of a tile lie in shared memory: rows of codes and of scales, `codes` and `scales` bytes apart.  All heads of
// a row come together, the scales behind the codes; some of them in two loads, the scales behind all codes of the tile.
struct Place4 {
    int32_t codes, scales;
    int32_t first;  // of the first row's scales
    int32_t bytes;  // of a tile
    int32_t apart;  // two loads
};

struct FewParams : Q4Params {
    int32_t bf16;
    int32_t unit_heads;        // key heads of a unit
    int32_t split;             // warps of a key head
    int32_t tile;              // keys
    int32_t slots;             // tiles of each ring
    int32_t piece_rows;        // slots that one TMA brings: they never leave a page
    Place4 kl, vl;
};

struct Aux {
    uint64_t k_full[kMaxSlots], k_empty[kMaxSlots], v_full[kMaxSlots], v_empty[kMaxSlots], sync;
    int scan[4 * 17];
    Place place;
    Walk walk[17];  // of each warp: held in registers it would crowd the loop over the tiles
    float m[16][16], l[16][16];  // of a warp's rows
    int answer;
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

// One tile of rows of keys or values: a TMA (two where heads are apart) for each run of slots inside a page, spread over the lanes.
// h0: the unit's first head; `ready` waits for the slot.
template <typename Ready>
__device__ __forceinline__ bool load_rows(const FewParams &p, const CUtensorMap *map, const CUtensorMap *scale_map, int dim, const Place4 &place,
                                          const int32_t *row, int kb, int lo, int hi, int h0, uint32_t to, uint32_t bar, const Ready &ready)
{
    const int lane = threadIdx.x & 31, pr = p.piece_rows;
    const int p0 = max(0, lo - kb) / pr, p1 = (min(hi - kb, p.tile) + pr - 1) / pr;
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
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)((p1 - p0) * pr) * (place.codes + (place.apart ? place.scales : 0)));
    __syncwarp();
    for (int i = p0 + lane; i < p1; i += 32) {
        if (i >= p0 + 32) find(i);
        tma_load_3d(to + i * pr * place.codes, map, bar, h0 * dim / 8, slot, page);
        if (place.apart)
            tma_load_3d(to + place.first + i * pr * place.scales, scale_map, bar, ((p.heads_all * dim / 2 + h0 * dim / 16) & ~15) / 4, slot, page);
    }
    __syncwarp();
    return true;
}

// Pieces (O [head, row][D], then a maximum and a sum a row) of rows that some part holds, for join_pieces.
struct Q4Pieces {
    const float *first;  // the first piece
    int64_t second;      // floats from it to the second one
    int64_t apart;       // between the others
    int count;
    __device__ __forceinline__ const float *operator()(int i) const { return first + (i == 0 ? 0 : second + (i - 1) * apart); }
};

// Four columns of a row of all pieces, in their order: eight pieces' loads in flight.
template <int D>
__device__ __forceinline__ float4 join_pieces(const Q4Pieces &at, int row, int quad, int stats, float &top, float &sum)
{
    top = -INFINITY, sum = 0.0f;
#pragma unroll 8
    for (int i = 0; i < at.count; i++) top = fmaxf(top, __ldcg(at(i) + stats + 2 * row));
    const float z = top == -INFINITY ? 0.0f : top;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int i0 = 0; i0 < at.count; i0 += 8) {
        float4 x[8];
        float2 ml[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f), ml[i] = make_float2(-INFINITY, 0.0f);
            if (i0 + i < at.count) {
                x[i] = __ldcg(reinterpret_cast<const float4 *>(at(i0 + i) + row * D) + quad);
                ml[i] = __ldcg(reinterpret_cast<const float2 *>(at(i0 + i) + stats + 2 * row));
            }
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float a = exp2_fast(ml[i].x - z);
            sum += ml[i].y * a;
            v.x += x[i].x * a, v.y += x[i].y * a, v.z += x[i].z * a, v.w += x[i].w * a;
        }
    }
    return v;
}

// H: the unit's heads where they are all of a row's and fill the widths D, and pages have runs of four slots or more (rows then lie
// a constant distance apart), else 0.
template <int D, int NT, int H>
__global__ void __launch_bounds__(Few<D, NT>::kThreads, 1)
attention_q4_few_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap ks_map,
                        const __grid_constant__ CUtensorMap vs_map, const __grid_constant__ FewParams p)
{
    using F = Few<D, NT>;
    extern __shared__ __align__(128) unsigned char smem[];
    Aux &aux = *reinterpret_cast<Aux *>(smem);
    float *const joins = reinterpret_cast<float *>(smem + ((sizeof(Aux) + 127) & ~127u));
    const uint32_t ring = smem_addr(joins) + ((F::kJoin + 127) & ~127u);
    const uint32_t v_ring = ring + (uint32_t)p.slots * p.kl.bytes;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const Batch &b = p.b;
    const Waiter wait{&aux.gave_up, b.err};
    const bool bf16 = p.bf16;
    const int heads = H ? H : p.unit_heads, split = H ? F::kWarps / H : p.split, users = heads * split;  // warps that compute: users
    const int dk = H ? D : p.k.dim, dv = H ? D : p.v.dim, tile_keys = 16 * split * F::kSteps;
    constexpr uint32_t kPitch = Few<D, NT>::pitch(H);
    const uint32_t k_row = H ? kPitch : p.kl.codes, y_row = H ? kPitch : p.kl.scales, v_row = H ? kPitch : p.vl.codes, x_row = H ? kPitch : p.vl.scales;
    const uint32_t k_tile = H ? kPitch * tile_keys : p.kl.bytes, v_tile = H ? kPitch * tile_keys : p.vl.bytes;

    if (tid == 0) {
        aux.gave_up = 0;
        for (int i = 0; i < p.slots; i++) {
            mbar_init(smem_addr(&aux.k_full[i]), 1);
            mbar_init(smem_addr(&aux.v_full[i]), 1);
            mbar_init(smem_addr(&aux.k_empty[i]), users);
            mbar_init(smem_addr(&aux.v_empty[i]), users);
        }
        mbar_init(smem_addr(&aux.sync), users);
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
    } else if (warp == 0) {
        // ---- rows of keys and values ----
        int it = 0;
        bool ok = true;
        do {
            const int32_t *row = p.table + (int64_t)w.at.req * p.table_stride;
            const int h0 = w.at.head * heads;
            for (int t = 0; ok && t < w.n && w.u.tiles > 0; t++, it++) {
                const int s = it % p.slots, kb = (w.u.tile0 + w.at.off + t) << b.tile_shift;
                const uint32_t phase = (uint32_t)(it / p.slots - 1) & 1;
                ok = load_rows(p, &k_map, &ks_map, p.k.dim, p.kl, row, kb, w.u.lo, w.u.hi, h0, ring + s * p.kl.bytes, smem_addr(&aux.k_full[s]),
                               [&] { return it < p.slots || wait.warp(smem_addr(&aux.k_empty[s]), phase); }) &&
                     load_rows(p, &v_map, &vs_map, p.v.dim, p.vl, row, kb, w.u.lo, w.u.hi, h0, v_ring + s * p.vl.bytes, smem_addr(&aux.v_full[s]),
                               [&] { return it < p.slots || wait.warp(smem_addr(&aux.v_empty[s]), phase); });
            }
            __syncwarp();
            if (ok) ok = next_of(w, b);
            __syncwarp();
        } while (ok);
    } else if (warp <= users) {
        const int me = warp - 1, h = me / split, part = me - h * split;
        bool ok = true;
        const int n = lane >> 2, t = lane & 3;
        const uint32_t rk = (kOrder >> (4 * n)) & 7;                                            // keys of score rows n, n + 8
        const uint32_t ra = (kOrder >> (8 * t)) & 7, rb = (kOrder >> (8 * t + 4)) & 7;          // keys of product columns 2 t, 2 t + 1
        const uint32_t g0 = 16u * part;
        // this thread's scales in a word of them; dimensions that heads do not have count as zeros
        const uint32_t k_mask = t * (D / 4) >= dk ? 0u : D == 128 && t * (D / 4) + 16 < dk ? 0xffffu : 0xffu;
        const uint32_t v_mask = n * (D / 8) < dv ? 0xffu : 0u;
        int it = 0, syncs = 0;
        const auto sync_all = [&] {
            warp_arrive(smem_addr(&aux.sync));
            ok = wait.warp(smem_addr(&aux.sync), syncs++ & 1);
            return ok;
        };
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
            uint32_t qf[NT][D / 16][2];
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
                float to = 1.0f, back = 1.0f;
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
                    const uint32_t e = min(max(__float_as_uint(most) >> 23, 1u), 253u);
                    to = __uint_as_float((254u - e) << 23);
                    back = __uint_as_float(e << 23);
                }
#pragma unroll
                for (int i = 0; i < D / 32; i++) {
                    const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        qf[x][2 * i + (j >> 1)][j & 1] =
                            bf16 ? pack2<false>(__uint_as_float(v[j] << 16) * to, __uint_as_float(v[j] & 0xffff0000u) * to) : v[j];
                }
#pragma unroll
                for (int i = 0; i < 2; i++)  // a normal number: a hidden score, -inf, stays that in the product with it
                    c[x][i] = fminf(fmaxf(p.o.c * __shfl_sync(0xffffffffu, back, (2 * t + i) * 4), 0x1p-126f), 0x1p127f);
            }
            float o[D / 16][NT][4];
            float m[NT][2], l[NT][2];
#pragma unroll
            for (int x = 0; x < NT; x++) {
#pragma unroll
                for (int i = 0; i < D / 16; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) o[i][x][j] = 0.0f;
                m[x][0] = m[x][1] = -INFINITY;
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
            const auto work = [&](auto hide, int kb, int s, uint32_t phase) {
                constexpr bool kHide = decltype(hide)::value;
                const auto unseen = [&](int key) { return key < seen_lo || key >= seen_hi; };
                if (!wait.warp(smem_addr(&aux.k_full[s]), phase)) return false;
                // ---- scores: S^T of 16 keys by 8 rows a step ----
                const uint32_t kp = k_at + s * k_tile, yp = y_at + s * k_tile;
                float sc[F::kSteps][NT][4];
#pragma unroll
                for (int step = 0; step < F::kSteps; step++) {
#pragma unroll
                    for (int x = 0; x < NT; x++)
#pragma unroll
                        for (int j = 0; j < 4; j++) sc[step][x][j] = 0.0f;
                    const uint32_t r0 = kp + step * 16 * split * k_row, r1 = r0 + 8 * k_row;
                    const uint32_t y0 = yp + step * 16 * split * y_row, y1 = y0 + 8 * y_row;
                    uint32_t w0[D / 32], w1[D / 32], u0, u1;
                    if (D == 128) {
                        const uint4 a = ld_smem16(r0), d = ld_smem16(r1);
                        w0[0] = a.x, w0[1] = a.y, w0[D / 32 - 2] = a.z, w0[D / 32 - 1] = a.w;
                        w1[0] = d.x, w1[1] = d.y, w1[D / 32 - 2] = d.z, w1[D / 32 - 1] = d.w;
                        u0 = ld_smem2(y0), u1 = ld_smem2(y1);
                    } else {
                        const uint2 a = ld_smem8(r0), d = ld_smem8(r1);
                        w0[0] = a.x, w0[1] = a.y, w1[0] = d.x, w1[1] = d.y;
                        u0 = ld_smem1(y0), u1 = ld_smem1(y1);
                    }
                    if (!H) u0 &= k_mask, u1 &= k_mask;
                    if (kHide) {  // what no row sees counts as zeros: it may hold anything
                        const int key = kb + (int)(g0 + 16 * split * step + rk);
                        if (unseen(key)) u0 = 0;
                        if (unseen(key + 8)) u1 = 0;
                    }
                    u0 = e4m3x2_to_f16(u0), u1 = e4m3x2_to_f16(u1);
#pragma unroll
                    for (int i = 0; i < D / 32; i++) {
                        const uint32_t z0 = prmt(u0, u0, i < 2 ? 0x1010 : 0x3232), z1 = prmt(u1, u1, i < 2 ? 0x1010 : 0x3232);
                        uint32_t a[4], d[4];
                        q4_to_f16(w0[i], a);
                        q4_to_f16(w1[i], d);
#pragma unroll
                        for (int j = 0; j < 4; j++) a[j] = mul_f16x2(a[j], z0), d[j] = mul_f16x2(d[j], z1);
#pragma unroll
                        for (int j = 0; j < 2; j++)
#pragma unroll
                            for (int x = 0; x < NT; x++) mma16816(sc[step][x], a[2 * j], d[2 * j], a[2 * j + 1], d[2 * j + 1], qf[x][2 * i + j][0], qf[x][2 * i + j][1]);
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
                        top[x][i] = v * c[x][i];
                        grow |= top[x][i] > m[x][i] + 8.0f;
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
                            const float a = now == -INFINITY ? 1.0f : exp2_fast(m[x][i] - now);
                            m[x][i] = now;
                            l[x][i] *= a;
#pragma unroll
                            for (int k = 0; k < D / 16; k++) o[k][x][i] *= a, o[k][x][i + 2] *= a;
                        }
                }
                uint32_t pf[F::kSteps][NT][2];
#pragma unroll
                for (int x = 0; x < NT; x++) {
                    const float off0 = m[x][0] == -INFINITY ? 0.0f : 7.0f - m[x][0], off1 = m[x][1] == -INFINITY ? 0.0f : 7.0f - m[x][1];
#pragma unroll
                    for (int step = 0; step < F::kSteps; step++) {
                        float e[4];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            e[j] = exp2_fast(fmaf(sc[step][x][j], c[x][j & 1], j & 1 ? off1 : off0));
                            l[x][j & 1] += e[j];
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
            for (int tile = 0; ok && tile < tiles; tile++, it++) {
                const int s = it % p.slots, kb = key0 + tile * tile_keys;
                const uint32_t phase = (uint32_t)(it / p.slots) & 1;
                if (kb < clean_lo || kb + tile_keys > clean_hi)
                    ok = work(std::true_type(), kb, s, phase);
                else
                    ok = work(std::false_type(), kb, s, phase);
            }
            if (!ok) break;
            // ---- the warps of a head join ----
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    float v = l[x][i];
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
                    const int r = 8 * x + 2 * t + i;
                    if (n == 0) aux.m[me][r] = m[x][i], aux.l[me][r] = v;
                    float4 *to = reinterpret_cast<float4 *>(joins + (me * F::kRows + r) * F::kPitch + n * (D / 8));
#pragma unroll
                    for (int k = 0; k < D / 32; k++) to[k] = make_float4(o[2 * k][x][i], o[2 * k][x][i + 2], o[2 * k + 1][x][i], o[2 * k + 1][x][i + 2]);
                }
            if (!sync_all()) break;
            const bool whole = w.whole();
            const auto row_out = [&](int hh, int r, int64_t &lse_at) {
                int g;
                const int64_t token = token_of(r, g);
                const int head = (head0 + hh) * (int)b.group.d + g;
                lse_at = token * p.o.heads + head;
                return p.o.out + token * p.o.out_token + (int64_t)head * p.o.out_head;
            };
            // (O, m, l) of a row as the caller wants it: to the output, or to a fragment [head, row][D], m, l
            const auto finish = [&](int hh, int r, int quad, float4 v, float top, float sum, float *frag) {
                if (frag != nullptr) {
                    const int at = hh * F::kRows + r;
                    __stcg(reinterpret_cast<float4 *>(frag + at * D) + quad, v);
                    if (quad == 0) {
                        __stcg(frag + heads * F::kRows * D + 2 * at, top);
                        __stcg(frag + heads * F::kRows * D + 2 * at + 1, sum);
                    }
                    return;
                }
                int64_t lse_at;
                char *to = row_out(hh, r, lse_at);
                const float inv = sum > 0.0f ? p.v_scale / sum : 0.0f;
                if (quad * 4 < p.o.dv) {
                    uint2 z;
                    z.x = bf16 ? pack2<true>(v.x * inv, v.y * inv) : pack2<false>(v.x * inv, v.y * inv);
                    z.y = bf16 ? pack2<true>(v.z * inv, v.w * inv) : pack2<false>(v.z * inv, v.w * inv);
                    *reinterpret_cast<uint2 *>(to + quad * 8) = z;
                }
                if (quad == 0 && p.o.lse) p.o.lse[lse_at] = sum > 0.0f ? fmaf(top, 0.69314718055994530942f, weight_log<false>(sum)) : -INFINITY;
            };
            float *const mine = p.ws + (int64_t)(2 * blockIdx.x + (w.at.off == 0 ? 1 : 0)) * (256 * 130);
            for (int i = me * 32 + lane; i < heads * rows * (D / 4); i += users * 32) {
                const int quad = i % (D / 4), hr = i / (D / 4), hh = hr / rows, r = hr - hh * rows;
                float top = -INFINITY, sum = 0.0f;
                for (int k = 0; k < split; k++) top = fmaxf(top, aux.m[hh * split + k][r]);
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int k = 0; k < split; k++) {
                    const int at = hh * split + k;
                    const float a = top == -INFINITY ? 0.0f : exp2_fast(aux.m[at][r] - top);
                    const float4 x = *reinterpret_cast<const float4 *>(joins + (at * F::kRows + r) * F::kPitch + 4 * quad);
                    sum += aux.l[at][r] * a;
                    v.x += x.x * a, v.y += x.y * a, v.z += x.z * a, v.w += x.w * a;
                }
                finish(hh, r, quad, v, top, sum, whole ? nullptr : mine);
            }
            if (!whole) {
                // ---- the CTA that finishes a cut unit's last piece joins them, in the order of the keys; of many pieces the last of
                // every kSum (3 to 10 at the unit's end) adds those up first, as in kv_attention.cuh ----
                const Cut cut(line, w.pos - w.at.off, unit_cost(w.u));
                const bool many = cut.count > kSum + kSum / 2;
                const int sums = (cut.count - 3) / kSum + 1, mine_of = min(cut.nth / kSum, sums - 1);
                const auto slot = [&](int piece, int odd) { return p.ws + (int64_t)(2 * (cut.c0 + piece) + odd) * (256 * 130); };
                for (bool sum = many;; sum = false) {
                    const int from = sum ? mine_of * kSum : 0, count = sum ? (mine_of + 1 < sums ? kSum : cut.count - from) : many ? sums : cut.count;
                    __threadfence();
                    if (!sync_all()) break;
                    if (me == 0 && lane == 0) {
                        int *counter = p.counters + 2 * (cut.c0 + (sum ? 1 + mine_of : 0));
                        const bool last = atomicAdd(counter, 1) == count - 1;
                        if (last) atomicExch(counter, 0);  // as the next call wants it
                        __threadfence();
                        *(volatile int *)&aux.answer = last;
                    }
                    if (!sync_all()) break;
                    if (!*(volatile int *)&aux.answer) break;
                    const bool of_sums = many && !sum;
                    Q4Pieces at;  // pieces lie in even slots but the unit's first, sums in the odd slot of their second piece
                    at.count = count;
                    at.first = of_sums ? slot(1, 1) : slot(from, from == 0);
                    at.apart = (int64_t)(of_sums ? kSum : 1) * 2 * (256 * 130);
                    at.second = of_sums ? at.apart : slot(from + 1, 0) - at.first;
                    for (int i = me * 32 + lane; i < heads * rows * (D / 4); i += users * 32) {
                        const int quad = i % (D / 4), hr = i / (D / 4), hh = hr / rows, r = hr - hh * rows;
                        float top, total;
                        const float4 v = join_pieces<D>(at, hh * F::kRows + r, quad, heads * F::kRows * D, top, total);
                        finish(hh, r, quad, v, top, total, sum ? slot(from + 1, 1) : nullptr);
                    }
                    if (!sum) break;
                }
                if (!ok) break;
            }
            if (!sync_all()) break;  // the next unit writes to the join's place
        } while (next_unit());
    }
    // common exit
    __syncwarp();
    __syncthreads();
    if (aux.gave_up) {  // let copies in flight land before the shared memory is given back
        const unsigned long long t0 = now_ns();
        while (now_ns() - t0 < 10000000ull) {}
    }
}

template <int D, int NT, int H>
int launch_kernel(const CUtensorMap *map, const FewParams &p, const DeviceInfo *dev, uint32_t bytes, cudaStream_t s)
{
    const auto kernel = attention_q4_few_kernel<D, NT, H>;
    if (dev == nullptr) {
        const int st = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
        return st != KV_OK ? st : load_kernels(kernel);
    }
    return cuda_status(launch(kernel, dim3(dev->num_sms), dim3(Few<D, NT>::kThreads), bytes, s, map[0], map[1], map[2], map[3], p));
}

// dev: null to prepare the kernels.
template <int D, int NT>
int launch_few(FewParams &p, const DeviceInfo *dev, cudaStream_t s)
{
    using F = Few<D, NT>;
    constexpr uint32_t kFixed = ((sizeof(Aux) + 127) & ~127u) + ((F::kJoin + 127) & ~127u), kAll = 227 * 1024;
    CUtensorMap map[4];
    if (dev == nullptr) {
        const int st = launch_kernel<D, NT, 0>(map, p, dev, kAll, s);
        return st != KV_OK ? st : launch_kernel<D, NT, 8>(map, p, dev, kAll, s);
    }
    const int all = p.heads_all;
    int heads = all < kMaxHeads ? all : kMaxHeads;
    while (all % heads) heads--;
    int split = 1;
    while (2 * split * heads <= F::kWarps) split *= 2;
    p.unit_heads = heads;
    p.split = split;
    p.tile = 16 * split * F::kSteps;
    p.piece_rows = piece_rows(p.k.desc->block_size, p.tile < 256 ? p.tile : 256);
    // A run of rows ends on a multiple of 128 bytes, where a TMA may begin; its rows lie 32 or 96 bytes off one where that allows it.
    const auto pitch = [&](int bytes) {
        const int step = p.piece_rows >= 4 ? 64 : 128 / p.piece_rows, off = p.piece_rows >= 4 ? 32 : 0;
        return (bytes - off + step - 1) / step * step + off;
    };
    const auto place = [&](int dim) {
        Place4 l = {};
        const int codes = heads * dim / 2;
        l.apart = heads < all;
        if (l.apart) {
            l.codes = pitch(codes);
            l.scales = pitch((heads * dim / 16 + 14 + 15) / 16 * 16);
            l.first = p.tile * l.codes;
            l.bytes = p.tile * (l.codes + l.scales);
        } else {
            l.codes = l.scales = pitch((int)q4_row_bytes(heads, dim));
            l.first = codes;
            l.bytes = p.tile * l.codes;
        }
        return l;
    };
    p.kl = place(p.k.dim);
    p.vl = place(p.v.dim);
    const uint32_t pair = (uint32_t)(p.kl.bytes + p.vl.bytes);
    p.slots = (int)((kAll - kFixed - 128) / pair);
    if (p.slots > kMaxSlots) p.slots = kMaxSlots;
    if (p.slots < 1) return KV_ERR_UNSUPPORTED;
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
    const uint32_t bytes = kFixed + 128 + p.slots * pair;
    const bool plain = heads == 8 && all == 8 && p.k.dim == D && p.v.dim == D && p.piece_rows >= 4;
    return plain ? launch_kernel<D, NT, 8>(map, p, dev, bytes, s) : launch_kernel<D, NT, 0>(map, p, dev, bytes, s);
}

}  // namespace

// rows: of a unit, 8 or 16.
int run_q4_few(bool bf16, const Q4Params &q, const kv_attn_batch *batch, int rows, const DeviceInfo &dev, cudaStream_t s)
{
    FewParams p = {};
    static_cast<Q4Params &>(p) = q;
    p.bf16 = bf16;
    if (p.k.dim <= 64 && p.v.dim <= 64) return rows <= 8 ? launch_few<64, 1>(p, &dev, s) : launch_few<64, 2>(p, &dev, s);
    return rows <= 8 ? launch_few<128, 1>(p, &dev, s) : launch_few<128, 2>(p, &dev, s);
}

int preload_q4_few_kernels()
{
    FewParams p = {};
    for (int (*prepare)(FewParams &, const DeviceInfo *, cudaStream_t) : {launch_few<64, 1>, launch_few<64, 2>, launch_few<128, 1>, launch_few<128, 2>}) {
        const int st = prepare(p, nullptr, nullptr);
        if (st != KV_OK) return st;
    }
    return KV_OK;
}

}  // namespace pkv
