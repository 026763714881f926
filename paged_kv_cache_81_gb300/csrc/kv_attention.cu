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

#include "kv_attention_kernel.cuh"

namespace pkv {

namespace {

template <int DK, int DV, bool Bf16>
int launch_attention(const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const AttentionParams &p, int parts, cudaStream_t s, bool prepare)
{
    const auto kernel = attention_kernel<DK, DV, Bf16, NoRows>;
    if (prepare)
        return cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<DK, DV>::kBytes));
    return cuda_status(launch(kernel, dim3(parts), dim3(kThreads), Shape<DK, DV>::kBytes, s, qm, km, vm, p));
}

template <bool Bf16>
int pick_attention(int dk, int dv, const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const AttentionParams &p, int parts, cudaStream_t s, bool prepare)
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
    AttentionParams p = {};
    CUtensorMap m;
    for (int dk : {64, 128, 192})
        for (bool bf : {false, true}) {
            const int st = bf ? pick_attention<true>(dk, dk == 64 ? 64 : 128, m, m, m, p, 0, nullptr, true)
                              : pick_attention<false>(dk, dk == 64 ? 64 : 128, m, m, m, p, 0, nullptr, true);
            if (st != KV_OK) return st;
        }
    return load_kernels(attention_kernel<64, 64, false, NoRows>, attention_kernel<64, 64, true, NoRows>, attention_kernel<128, 128, false, NoRows>,
                        attention_kernel<128, 128, true, NoRows>, attention_kernel<192, 128, false, NoRows>, attention_kernel<192, 128, true, NoRows>);
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
    AttentionParams p = {};
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
