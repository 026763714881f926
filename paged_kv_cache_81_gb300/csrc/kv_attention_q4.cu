// kv_attention_q4: attention over a 4-bit cache, its checks and the choice of its kernel.
#include <cmath>

#include "kv_attention_q4.cuh"

namespace pkv {

int preload_q4_kernels()
{
    int st = preload_q4_few64_kernels();
    if (st == KV_OK) st = preload_q4_few128_kernels();
    return st != KV_OK ? st : preload_q4_many_kernels();
}

}  // namespace pkv

using namespace pkv;

extern "C" {

int kv_attention_q4(const kv_attn_desc *d, const kv_attn_batch *batch, const kv_cache_desc *k, int32_t k_tensor, int32_t k_plane,
                    const kv_cache_desc *v, int32_t v_tensor, int32_t v_plane, float k_scale, float v_scale, const void *q, int64_t q_token_stride,
                    int64_t q_head_stride, void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                    int64_t workspace_bytes, kv_stream_t stream)
{
    if (d == nullptr || d->n_heads <= 0 || d->n_kv_heads <= 0 || d->n_heads % d->n_kv_heads != 0 || d->head_dim <= 0 || d->head_dim_v <= 0 ||
        d->window < 0 || !good_scale(d->scale) || !good_scale(k_scale) || !good_scale(v_scale) || !good_scale(d->scale * k_scale) ||
        (d->dtype != KV_BF16 && d->dtype != KV_F16))
        return KV_ERR_INVALID_ARG;
    int st = check_batch(batch);
    if (st != KV_OK) return st;
    const int group = d->n_heads / d->n_kv_heads;
    if (d->head_dim % 32 || d->head_dim_v % 32) return KV_ERR_ALIGN;
    if (group > 128 || (d->window && !d->causal)) return KV_ERR_UNSUPPORTED;
    if ((st = check_q4_plane(k, k_tensor, k_plane, d->n_kv_heads, d->head_dim)) != KV_OK) return st;
    if ((st = check_q4_plane(v, v_tensor, v_plane, d->n_kv_heads, d->head_dim_v)) != KV_OK) return st;
    if (k->block_size != v->block_size) return KV_ERR_INVALID_ARG;
    if (batch->n_reqs == 0 || batch->n_tokens == 0) return KV_OK;
    if ((st = check_rows(q, q_token_stride, q_head_stride)) != KV_OK) return st;
    if ((st = check_rows(out, out_token_stride, out_head_stride)) != KV_OK) return st;
    if (workspace == nullptr) return KV_ERR_INVALID_ARG;
    if (!aligned16(workspace) || ((uintptr_t)lse & 3u)) return KV_ERR_ALIGN;
    // By the rows (tokens times query heads of a key head) that a request has on average.  Each side measured, 16 requests of 8000 with 8 key
    // heads of 128 in bf16, groups of 4: 8 rows in units of 8 46 us, of 16 57; 16 rows with few rows' kernel 66, many rows' 104; 20 rows 93 and 106;
    // 32 rows 96 and 106; 36 rows 122 and 111.  (64 requests of 2000: 32 rows 94 and 127, 48 rows 133 and 131; one of 120000: 32 rows 104 and 105.)
    // One kernel a call: 200 decoding requests of 1000 to 4000 take 114 us, a chunk of 1024 tokens over 8192 135 (of 4096 368), in one call 681 (806).
    const bool many = batch->n_tokens * group > 32ll * batch->n_reqs;
    const int rows = batch->n_tokens * group <= 8ll * batch->n_reqs ? 8 : 16;
    Q4Params p = {};
    if ((st = fill_batch(&p.b, batch, d->n_heads, d->n_kv_heads, k->block_size, many ? q4_unit_rows(group) : group > rows ? rows : rows / group * group,
                         many ? q4_tile_shift() : 5, d->causal, d->window)) != KV_OK)
        return st;
    const DeviceInfo *dev = current_device();
    if (dev == nullptr) return KV_ERR_CUDA;
    if (workspace_bytes < attention_workspace(dev->num_sms)) return KV_ERR_RANGE;
    if ((st = prepare_attention_q4(*dev)) != KV_OK) return st;
    p.b.err = dev->err_word;
    const auto plane = [](const kv_cache_desc *c, int tensor, int which, int dim) {
        return Q4Plane{c->base[tensor] + (which ? (uint64_t)c->plane_stride : 0), c, dim};
    };
    p.k = plane(k, k_tensor, k_plane, d->head_dim);
    p.v = plane(v, v_tensor, v_plane, d->head_dim_v);
    p.table = batch->block_table;
    p.table_stride = batch->bt_row_stride;
    p.num_blocks = (int32_t)(k->num_blocks < v->num_blocks ? k->num_blocks : v->num_blocks);
    p.no_page = (int32_t)(k->num_blocks < v->num_blocks ? v->num_blocks : k->num_blocks);
    p.block = make_fastdiv((uint32_t)k->block_size);
    p.q = (const char *)q;
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.heads_all = d->n_kv_heads;
    const float scale = d->scale * k_scale;
    p.o = Output{(char *)out, out_token_stride, out_head_stride, lse, d->n_heads, d->head_dim_v, scale, scale * kLog2e};
    p.v_scale = v_scale;
    p.counters = (int *)workspace;
    p.ws = (float *)((char *)workspace + kCounterBytes);
    if (many) return run_q4_many(d->dtype == KV_BF16, p, batch, *dev, (cudaStream_t)stream);
    const auto few = d->head_dim <= 64 && d->head_dim_v <= 64 ? run_q4_few64 : run_q4_few128;
    return few(d->dtype == KV_BF16, p, rows, *dev, (cudaStream_t)stream);
}

}  // extern "C"
