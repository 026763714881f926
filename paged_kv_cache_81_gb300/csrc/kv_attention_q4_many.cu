// kv_attention_q4 for many rows: prefill chunks, and decoding of more than 32 query rows a key head.
//
// kv_attention's kernel (kv_attention.cu) with tiles of fp16 keys and values that four warps make of packed rows, which come by
// TMA: a head's codes and the 16 bytes that hold its scales.  A thread takes 32 elements of a row (16 bytes of codes, two scales) at a
// time and writes them as four 16-byte pieces of the swizzled panels, one conversion and one product a pair: a code times its scale is
// exact in fp16, so the products are those of the values that the cache stands for.  bf16 queries are brought to fp16 as well, a
// power of two a row apart; made into bf16 instead, through 32-bit products, tiles took 870 us where they take 811 now, and weights lost three bits.
//
// Four chunks of 2048 to 4096 tokens over 4096 to 8192, 32 heads over 8 of 128: 811 us (fp16 789), 1.1 PFLOP/s; kv_attention over 16-bit rows
// 670.  The warps that make tiles take issue slots and shared memory from the softmax, so that a step takes a fifth more than there.
// Their loop is short: straight code for all rows of a tile runs at the rate that instructions come at (870, 1041 us).
#define PKV_APART __forceinline__

#include "kv_attention_kernel.cuh"
#include "kv_attention_q4.cuh"

namespace pkv {

namespace {

// A plane of packed rows.  In the stage: a tile's codes [key][codes bytes], then its pieces of scales [key][units bytes].
struct Q4Rows {
    CUtensorMap scale_map;
    int32_t dim, scales;         // of a head; where a row's scales begin
    int32_t codes, units;        // bytes a key in the stage
    int32_t stage_bytes;
    int32_t single;              // rows come one by one, by untiled copies from `base`
    uint32_t row_bytes;
    uint64_t base;
    int64_t block_stride, token_stride;

    // One tile's rows: two TMAs for each run of slots inside a page, spread over the lanes; `ready` waits for the slot.
    template <typename Ready>
    __device__ __forceinline__ bool load(const RowsParams<Q4Rows> &p, const CUtensorMap *map, const int32_t *row, int kb, int lo, int hi, int head, uint32_t to,
                                         uint32_t bar, bool report, const Ready &ready) const
    {
        const int lane = threadIdx.x & 31, pr = p.piece_rows;
        const int p0 = max(0, lo - kb) / pr, p1 = (min(hi - kb, kTile) + pr - 1) / pr;
        int page = 0, slot = 0;
        const auto find = [&](int i) {
            const uint32_t key = (uint32_t)(kb + i * pr), col = fdiv(key, p.block);
            slot = (int)(key - col * p.block.d);
            page = __ldg(row + col);
            if (page < 0 || page >= p.num_blocks) {
                if (report) set_error(p.b.err, KV_DERR_TABLE);
                page = p.no_page;
            }
        };
        if (p0 + lane < p1) find(p0 + lane);
        if (!ready()) return false;
        if (single) {
            const uint32_t unit_from = (uint32_t)((scales + head * (dim / 16)) & ~15), unit_bytes = min((uint32_t)units, row_bytes - unit_from);
            for (int i0 = p0; i0 < p1; i0 += 32) {
                const int i = i0 + lane;
                if (i0 > p0 && i < p1) find(i);
                const bool there = i < p1 && page != p.no_page;
                const uint32_t all = __ballot_sync(0xffffffffu, there);
                if (lane == 0) mbar_expect(bar, (uint32_t)__popc(all) * (codes + unit_bytes));
                __syncwarp();
                const uint32_t code_to = to + i * codes, unit_to = to + kTile * codes + i * units;
                if (there) {
                    const uint64_t from = base + (uint64_t)page * block_stride + (uint64_t)slot * token_stride;
                    bulk_load(code_to, from + (uint32_t)(head * codes), codes, bar);
                    bulk_load(unit_to, from + unit_from, unit_bytes, bar);
                } else if (i < p1) {
                    for (int x = 0; x < codes; x += 16) st_smem16(code_to + x, make_uint4(0, 0, 0, 0));
                    for (int x = 0; x < units; x += 16) st_smem16(unit_to + x, make_uint4(0, 0, 0, 0));
                }
            }
            warp_arrive(bar);
            return true;
        }
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)((p1 - p0) * pr) * (codes + units));
        __syncwarp();
        for (int i = p0 + lane; i < p1; i += 32) {
            if (i >= p0 + 32) find(i);
            tma_load_4d(to + i * pr * codes, map, bar, 0, head, slot, page);
            tma_load_3d(to + kTile * codes + i * pr * units, &scale_map, bar, ((scales + head * (dim / 16)) & ~15) / 4, slot, page);
        }
        __syncwarp();
        return true;
    }

    // A staged tile into panels, by 128 threads; rows outside [lo, hi) become zeros, whatever the stage holds there.
    template <int D>
    __device__ __forceinline__ void unpack(uint32_t stage, uint32_t tile, int head, int lo, int hi, int thread) const
    {
        constexpr int kParts = D / 32, kRowsATurn = 128 / kParts;
        const int part = thread % kParts, r0 = thread / kParts;
        // of four parts of a row the last two go the other way round, or they would meet the first two in the banks
        const int swap = kParts == 4 ? part & 2 : 0;
        const bool there = part * 32 < dim;
        const uint32_t code_at = stage + r0 * codes + part * 16;
        const uint32_t unit_at = stage + kTile * codes + r0 * units + ((scales + head * (dim / 16)) & 15) + part * 2;
        const uint32_t to = tile + (part >> 1) * kPanel + r0 * 128;
        uint32_t at[4];  // of the four pieces: the same in every turn, whose rows are a multiple of eight apart
#pragma unroll
        for (int i = 0; i < 4; i++) at[i] = to + ((((part & 1) * 4 + (i ^ swap)) ^ (r0 & 7)) << 4);
        const auto load = [&](int j, uint4 &c, uint32_t &u) {
            const int r = r0 + j * kRowsATurn;
            c = ld_smem16(code_at + j * kRowsATurn * codes);
            uint16_t two;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(two) : "r"(unit_at + j * kRowsATurn * units) : "memory");
            u = there && r >= lo && r < hi ? two : 0;
        };
        uint4 c, next_c;
        uint32_t unit, next_unit;
        load(0, next_c, next_unit);
        // a short loop: straight code for all rows runs at the rate that instructions come at
#pragma unroll 1
        for (int j = 0; j < kTile / kRowsATurn; j++) {
            c = next_c, unit = next_unit;
            if (j + 1 < kTile / kRowsATurn) load(j + 1, next_c, next_unit);
            uint32_t u = e4m3x2_to_f16(unit);
            if (swap) u = u >> 16 | u << 16;
            const uint32_t z[2] = {u << 16 | (u & 0xffffu), u >> 16 | (u & 0xffff0000u)};
            const uint32_t word[4] = {swap ? c.z : c.x, swap ? c.w : c.y, swap ? c.x : c.z, swap ? c.y : c.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                uint32_t v[4];
                q4_to_f16(word[i], v);
#pragma unroll
                for (int k = 0; k < 4; k++) v[k] = mul_f16x2(v[k], z[i >> 1]);
                st_smem16(at[i] + j * kRowsATurn * 128, make_uint4(v[0], v[1], v[2], v[3]));
            }
        }
    }
};

template <int D, bool Bf16>
int launch_many(const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const RowsParams<Q4Rows> &p, int parts, cudaStream_t s, bool prepare)
{
    const auto kernel = attention_kernel<D, D, Bf16, Q4Rows>;
    if (prepare) {
        const int st = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024));
        return st != KV_OK ? st : load_kernels(kernel);
    }
    return cuda_status(launch(kernel, dim3(parts), dim3(kRowsThreads), 227 * 1024, s, qm, km, vm, p));
}

}  // namespace

// x, or the next multiple of `of`, a power of two.
static int round_up(int x, int of) { return of <= 1 ? x : (x + of - 1) / of * of; }

int q4_unit_rows(int group) { return 2 * (128 / group) * group; }
int q4_tile_shift() { return kTileShift; }

int run_q4_many(bool bf16, const Q4Params &q, const kv_attn_batch *batch, const DeviceInfo &dev, cudaStream_t s)
{
    RowsParams<Q4Rows> p = {};
    const int group = (int)q.b.group.d;
    p.b = q.b;
    p.table = q.table;
    p.table_stride = q.table_stride;
    p.num_blocks = q.num_blocks;
    p.block = q.block;
    p.o = q.o;
    p.o.values = q.v_scale;
    p.ws = q.ws;
    p.counters = q.counters;
    p.no_page = q.no_page;
    p.piece_rows = piece_rows(q.k.desc->block_size, kTile);
    p.q_box = box_tokens(128 / group, batch);
    const bool small = q.k.dim <= 64 && q.v.dim <= 64;
    CUtensorMap qm, km, vm;
    int st;
    const auto rows = [&](const Q4Plane &plane, Q4Rows *r, CUtensorMap *map) {
        r->dim = plane.dim;
        r->scales = q.heads_all * plane.dim / 2;
        // runs of rows begin on multiples of 128 bytes; scales of heads of 96 may lie across a 16-byte boundary
        r->codes = round_up(small ? 32 : 64, 128 / p.piece_rows);
        r->units = round_up(16 % (plane.dim / 16) ? 32 : 16, 128 / p.piece_rows);
        if (!small && p.piece_rows == 1) {  // two stages of them would not fit
            r->single = 1;
            r->codes = plane.dim / 2;
            r->units = 16 % (plane.dim / 16) ? 32 : 16;
            r->row_bytes = (uint32_t)plane.desc->row_bytes;
            r->base = plane.base;
            r->block_stride = plane.desc->block_stride;
            r->token_stride = plane.desc->token_stride;
        }
        r->stage_bytes = kTile * (r->codes + r->units);
        const int st = make_q4_code_map(map, plane.base, plane.desc, q.heads_all, plane.dim, r->codes, p.piece_rows);
        return st != KV_OK ? st : make_row_map(&r->scale_map, plane.base, plane.desc, r->units, p.piece_rows);
    };
    if ((st = rows(q.k, &p.k, &km)) != KV_OK || (st = rows(q.v, &p.v, &vm)) != KV_OK) return st;
    const int stage = p.k.stage_bytes > p.v.stage_bytes ? p.k.stage_bytes : p.v.stage_bytes;
    p.k.stage_bytes = p.v.stage_bytes = stage;
    p.stages = (int)((small ? Shape<64, 64, true>::kStage : Shape<128, 128, true>::kStage) / stage);
    if (p.stages > 4) p.stages = 4;
    if (p.stages < 2) return KV_ERR_UNSUPPORTED;
    if ((st = make_q_map(&qm, q.q, q.q_token, q.q_head, q.k.dim, q.o.heads, batch->n_tokens, group, p.q_box)) != KV_OK) return st;
    if (small)
        return bf16 ? launch_many<64, true>(qm, km, vm, p, dev.num_sms, s, false) : launch_many<64, false>(qm, km, vm, p, dev.num_sms, s, false);
    return bf16 ? launch_many<128, true>(qm, km, vm, p, dev.num_sms, s, false) : launch_many<128, false>(qm, km, vm, p, dev.num_sms, s, false);
}

int preload_q4_many_kernels()
{
    RowsParams<Q4Rows> p = {};
    CUtensorMap m;
    for (int (*launch)(const CUtensorMap &, const CUtensorMap &, const CUtensorMap &, const RowsParams<Q4Rows> &, int, cudaStream_t, bool) :
         {launch_many<64, false>, launch_many<64, true>, launch_many<128, false>, launch_many<128, true>}) {
        const int st = launch(m, m, m, p, 0, nullptr, true);
        if (st != KV_OK) return st;
    }
    return KV_OK;
}

}  // namespace pkv
