// kv8.cuh — internal interface of the 8-bit paged cache: the batch planned on the
// device (batch_plan.cu), the quantising writes (kv8_write.cu) and the attention over
// e4m3 pages (kv8_attn.cu).  include/dllm.h is the public ABI.
#pragma once

#include "kernels.cuh"

namespace dllm {

constexpr int kErrNoPages = 16;      // DLLM_DEVERR_NO_PAGES
constexpr int kKv8Group = 16;        // token positions that share a scale
constexpr int kKv8Groups = kPage / kKv8Group;
constexpr int kKv8MaxExp = 60;       // scales are within 2^-60 .. 2^60

// ---- the batch plan
struct PlanArgs {
  const int32_t* seq_len;
  const int32_t* block_start;
  const int32_t* block_len;
  const int32_t* held;
  int32_t* held_out;
  int32_t* table;        // [batch][max_pages]
  int32_t* cu_block;
  int32_t* cu_seq;
  int32_t* ring;         // [num_pages]
  const int32_t* state;  // head, count
  int32_t* state_out;
  int32_t* row_slot;     // [cap_rows], nullable, as the next two
  int32_t* row_seq;
  int32_t* row_pos;
  int32_t* err;
  int32_t batch, max_pages, num_pages, max_seq_len, cap_rows, cap_seq;
};
cudaError_t launch_batch_plan(const PlanArgs& a, int num_sms, cudaStream_t stream);

// ---- the cache and its writes
struct Kv8Pools {
  uint8_t* k;      // e4m3 [P][Hkv][64][d]
  uint8_t* v;
  float* k_scale;  // [P][Hkv][4]
  float* v_scale;
  int32_t n_kv_heads;
};
struct Kv8WriteArgs {
  BatchArgs bt;    // num_pages: the smaller of the pools'
  Kv8Pools kv;
  const void* k_src;  // bf16: rows at the strides below, or (from_pool) [P][Hkv][64][d]
  const void* v_src;
  int64_t k_row, k_head, v_row, v_head;  // elements
  int32_t head_dim;
  bool from_pool;
};
cudaError_t launch_kv8_write(const Kv8WriteArgs& a, int num_sms, cudaStream_t stream);

// ---- the attention
struct Kv8AttnArgs {
  BatchArgs bt;
  Kv8Pools kv;
  const void* q;        // bf16 rows at q_row elements, [H][d]
  int64_t q_row;
  void* o;              // bf16 rows of [H][d]
  float* lse;           // fp32 rows of [H], nullable
  int32_t full_rows;    // rows at cu_seq[b] + s_b + i, else at cu_block[b] + i
  int32_t n_heads;
  int32_t head_dim;
  float scale_log2;     // softmax scale * log2(e)
  void* ws;
  int32_t whole_units;  // set by the launcher: units are not split over CTAs
};
size_t kv8_attention_workspace_bytes(int max_block_len, int n_heads, int n_kv_heads, int head_dim, int num_sms);
cudaError_t launch_kv8_attention(const Kv8AttnArgs& a, int num_sms, cudaStream_t stream);

}  // namespace dllm
