// What the attention kernels' host sides share: argument checks, the batch they pass on, the workspace.
#pragma once

#include "kv_plan.cuh"
#include "kv_tensor.cuh"

namespace pkv {

constexpr int64_t kPlaceBytes = 16384;  // where each CTA's piece begins: 16 bytes a CTA

// Two fragments a CTA: of 256 rows x (128 values + maximum + sum) for kv_attention, of 128 rows x (256
// values + maximum + sum) for each CTA of kv_latent_attention.
inline int64_t attention_workspace(int num_sms) { return kPlaceBytes + (int64_t)num_sms * 2 * 256 * (128 + 2) * 4; }

int check_batch(const kv_attn_batch *t);
int fill_batch(Batch *b, const kv_attn_batch *t, int heads, int kv_heads, int block_size, int unit_rows, int causal, int window, int *err);
int check_plane(const kv_cache_desc *c, int tensor, int plane, int heads, int dim);
int check_rows(const void *p, int64_t token_stride, int64_t head_stride);
int piece_rows(int block_size);

// Launch attributes of every attention kernel, set once per device (kv_runtime.cu).
int prepare_attention(const DeviceInfo &dev);
int preload_attention_kernels();  // kv_attention.cu

}  // namespace pkv
