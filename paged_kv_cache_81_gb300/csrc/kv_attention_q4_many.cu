// kv_attention_q4 for many rows: prefill chunks, and decoding of more than 16 query rows a key head.
//
// kv_attention's kernel (kv_attention.cu) with tiles of 16-bit keys and values that three warps make of the 4-bit rows: a thread takes
// 32 elements of a row (16 bytes of codes, two scales) straight from global memory, asked for a tile ahead, and writes them as four
// 16-byte pieces of the swizzled panels.  A code times its scale is exact in fp16 and in bf16, so the products are those of the values
// that the cache stands for.  fp16: one conversion and one product a pair.  bf16: the conversion gives fp16 pairs; moved three bits
// down, their exponents stand where bf16's do, 112 too low, and the product with the scale times 2^112 mends that, exactly.
#include "kv_attention_kernel.cuh"
#include "kv_attention_q4.cuh"

namespace pkv {

namespace {

// A thread takes one of a row's parts of 32 elements, of every 96 / parts-th row of a tile.
template <int D>
constexpr int kParts = D / 32;
template <int D>
constexpr int kItems = (kTile * kParts<D> + 95) / 96;

struct Q4Rows {
    const char *base;  // of this plane
    int64_t block_stride, token_stride;
    int32_t dim, scales;  // scales: where a row's begin

    // The pages of a thread's rows of a tile: -1 where a row is not seen or not there.
    template <int D>
    struct Pages {
        int page[kItems<D>], slot[kItems<D>];
        __device__ __forceinline__ void look(const RowsParams<Q4Rows> &p, const Walk &w, int kb, int thread)
        {
            const int32_t *const row = p.table + (int64_t)w.at.req * p.table_stride;
#pragma unroll
            for (int j = 0; j < kItems<D>; j++) {
                const int r = thread / kParts<D> + j * (96 / kParts<D>), key = kb + r;
                page[j] = -1, slot[j] = 0;
                if (r >= kTile || key < w.u.lo || key >= w.u.hi) continue;
                const uint32_t col = fdiv((uint32_t)key, p.block);
                slot[j] = (int)((uint32_t)key - col * p.block.d);
                page[j] = __ldg(row + col);
                if (page[j] < 0 || page[j] >= p.num_blocks) {
                    set_error(p.b.err, KV_DERR_TABLE);
                    page[j] = -1;
                }
            }
        }
    };

    template <int D>
    struct Raw {
        uint4 codes[kItems<D>];
        uint32_t unit[kItems<D>];  // two scales

        __device__ __forceinline__ void fetch(const Q4Rows &plane, const Pages<D> &pages, int head, int thread)
        {
            const int part = thread % kParts<D>;
            const char *const from = plane.base + (int64_t)head * (plane.dim / 2) + part * 16;
            const char *const scale = plane.base + plane.scales + (int64_t)head * (plane.dim / 16) + part * 2;
#pragma unroll
            for (int j = 0; j < kItems<D>; j++) {
                codes[j] = make_uint4(0, 0, 0, 0), unit[j] = 0;
                if (pages.page[j] < 0 || part * 32 >= plane.dim) continue;
                const int64_t at = pages.page[j] * plane.block_stride + pages.slot[j] * plane.token_stride;
                codes[j] = __ldg(reinterpret_cast<const uint4 *>(from + at));
                unit[j] = __ldg(reinterpret_cast<const uint16_t *>(scale + at));
            }
        }

        // Pairs of one scale as the products take them.
        template <bool Bf16>
        static __device__ __forceinline__ uint32_t times(uint32_t pair, uint32_t unit)
        {
            uint32_t v;
            if (Bf16)
                asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"((pair >> 3 & 0x0fff0fffu) | (pair & 0x80008000u)), "r"(unit));
            else
                v = mul_f16x2(pair, unit);
            return v;
        }

        // Into a tile's panels; rows that were left out become zeros.
        template <bool Bf16>
        __device__ __forceinline__ void put(uint32_t tile, int thread) const
        {
            const int part = thread % kParts<D>;
            // of four parts of a row the last two go the other way round, or they would meet the first two in the banks
            const int swap = kParts<D> == 4 ? part & 2 : 0;
#pragma unroll
            for (int j = 0; j < kItems<D>; j++) {
                const int r = thread / kParts<D> + j * (96 / kParts<D>);
                if (r >= kTile) break;
                uint32_t u = e4m3x2_to_f16(unit[j]), z[2];
                if (swap) u = u >> 16 | u << 16;
                if (Bf16) {
                    float lo, hi;
                    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(lo), "=f"(hi) : "r"(u));
                    lo *= 0x1p112f, hi *= 0x1p112f;
                    z[0] = pack2<true>(lo, lo), z[1] = pack2<true>(hi, hi);
                } else {
                    z[0] = u << 16 | (u & 0xffffu), z[1] = u >> 16 | (u & 0xffff0000u);
                }
                const uint4 c = codes[j];
                const uint32_t word[4] = {swap ? c.z : c.x, swap ? c.w : c.y, swap ? c.x : c.z, swap ? c.y : c.w};
                const uint32_t panel = tile + (part >> 1) * kPanel;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    uint32_t v[4];
                    q4_to_f16(word[i], v);
                    const uint32_t s = z[i >> 1];
                    st_smem16(panel + panel_off((uint32_t)r, (uint32_t)((part & 1) * 4 + (i ^ swap))),
                              make_uint4(times<Bf16>(v[0], s), times<Bf16>(v[1], s), times<Bf16>(v[2], s), times<Bf16>(v[3], s)));
                }
            }
        }
    };
};

template <int D, bool Bf16>
int launch_many(const CUtensorMap &qm, const RowsParams<Q4Rows> &p, int parts, cudaStream_t s, bool prepare)
{
    const auto kernel = attention_kernel<D, D, Bf16, Q4Rows>;
    if (prepare) {
        const int st = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<D, D>::kBytes));
        return st != KV_OK ? st : load_kernels(kernel);
    }
    return cuda_status(launch(kernel, dim3(parts), dim3(kThreads), Shape<D, D>::kBytes, s, qm, qm, qm, p));
}

}  // namespace

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
    p.q_box = box_tokens(128 / group, batch);
    const auto rows = [&](const Q4Plane &plane) {
        return Q4Rows{(const char *)plane.base, plane.desc->block_stride, plane.desc->token_stride, plane.dim, q.heads_all * plane.dim / 2};
    };
    p.k = rows(q.k);
    p.v = rows(q.v);
    CUtensorMap qm;
    const int st = make_q_map(&qm, q.q, q.q_token, q.q_head, q.k.dim, q.o.heads, batch->n_tokens, group, p.q_box);
    if (st != KV_OK) return st;
    if (q.k.dim <= 64 && q.v.dim <= 64)
        return bf16 ? launch_many<64, true>(qm, p, dev.num_sms, s, false) : launch_many<64, false>(qm, p, dev.num_sms, s, false);
    return bf16 ? launch_many<128, true>(qm, p, dev.num_sms, s, false) : launch_many<128, false>(qm, p, dev.num_sms, s, false);
}

int preload_q4_many_kernels()
{
    RowsParams<Q4Rows> p = {};
    CUtensorMap m;
    for (int (*launch)(const CUtensorMap &, const RowsParams<Q4Rows> &, int, cudaStream_t, bool) :
         {launch_many<64, false>, launch_many<64, true>, launch_many<128, false>, launch_many<128, true>}) {
        const int st = launch(m, p, 0, nullptr, true);
        if (st != KV_OK) return st;
    }
    return KV_OK;
}

}  // namespace pkv
