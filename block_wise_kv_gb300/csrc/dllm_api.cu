// dllm_api.cu — the C ABI declared in include/dllm.h: host-side validation,
// workspace sizing and the launch sequence of each entry point.  Every check
// runs before the first launch, so a rejected call launches nothing.
#include <math.h>
#include <stdint.h>

#include "dllm.h"
#include "kernels.cuh"
#include "kv8.cuh"
#include "layer_ops.cuh"

using namespace dllm;

namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;

bool aligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

dllm_status check_desc(const dllm_layer_desc* d) {
  if (d == nullptr) return DLLM_ERR_INVALID_ARGUMENT;
  if (d->head_dim != 64 && d->head_dim != 128) return DLLM_ERR_UNSUPPORTED;
  if (d->page_size != kPage) return DLLM_ERR_UNSUPPORTED;
  if (d->d_model <= 0 || d->n_heads <= 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (d->d_model % 64 != 0) return DLLM_ERR_UNSUPPORTED;
  if ((static_cast<int64_t>(d->n_heads) * d->head_dim) % 128 != 0) return DLLM_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d->n_heads) * d->head_dim * 3 > 65535 * 128) return DLLM_ERR_UNSUPPORTED;
  if (!(d->rope_theta > 0.f) || !isfinite(d->rope_theta)) return DLLM_ERR_INVALID_ARGUMENT;
  if (!(d->rms_eps >= 0.f) || !isfinite(d->rms_eps)) return DLLM_ERR_INVALID_ARGUMENT;
  if (!(d->softmax_scale >= 0.f) || !isfinite(d->softmax_scale)) return DLLM_ERR_INVALID_ARGUMENT;
  return DLLM_OK;
}

dllm_status check_batch(const dllm_batch* b) {
  if (b == nullptr || b->batch < 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (b->batch == 0) return DLLM_OK;
  if (b->batch > 65535) return DLLM_ERR_UNSUPPORTED;
  if (!aligned(b->block_table, 4) || !aligned(b->seq_len, 4) || !aligned(b->block_start, 4) ||
      !aligned(b->block_len, 4) || !aligned(b->cu_block, 4) || !aligned(b->cu_seq, 4))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (b->error_flag != nullptr && !aligned(b->error_flag, 4)) return DLLM_ERR_INVALID_ARGUMENT;
  if (b->max_pages_per_seq < 1 || b->max_seq_len < 1 || b->max_block_len < 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (b->max_block_len > b->max_seq_len) return DLLM_ERR_INVALID_ARGUMENT;
  if (static_cast<int64_t>(b->max_pages_per_seq) * kPage < b->max_seq_len) return DLLM_ERR_INVALID_ARGUMENT;
  if (b->max_seq_len > 65535 * kPage) return DLLM_ERR_UNSUPPORTED;
  if (b->total_block_rows < 0 || b->total_seq_rows < 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (static_cast<int64_t>(b->total_block_rows) > static_cast<int64_t>(b->batch) * b->max_block_len)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (static_cast<int64_t>(b->total_seq_rows) > static_cast<int64_t>(b->batch) * b->max_seq_len)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (b->total_block_rows > b->total_seq_rows) return DLLM_ERR_INVALID_ARGUMENT;
  return DLLM_OK;
}

dllm_status check_cache(const dllm_cache* c, const dllm_layer_desc* d, bool need_q, bool need_state) {
  if (c == nullptr || c->num_pages < 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (static_cast<int64_t>(c->num_pages) * d->n_heads * kPage > kMaxRows) return DLLM_ERR_UNSUPPORTED;
  if (!aligned(c->k_pool, 16) || !aligned(c->v_pool, 16)) return DLLM_ERR_INVALID_ARGUMENT;
  if (need_q && !aligned(c->q_pool, 16)) return DLLM_ERR_INVALID_ARGUMENT;
  if (need_state && (!aligned(c->m_pool, 16) || !aligned(c->l_pool, 16) || !aligned(c->o_pool, 16)))
    return DLLM_ERR_INVALID_ARGUMENT;
  return DLLM_OK;
}

// The prefix state pools: all unset (0), all set and aligned (1), else invalid (-1).
int pre_pools(const dllm_cache* c) {
  if (c->m_pre == nullptr && c->l_pre == nullptr && c->o_pre == nullptr) return 0;
  if (!aligned(c->m_pre, 16) || !aligned(c->l_pre, 16) || !aligned(c->o_pre, 16)) return -1;
  return 1;
}

int device_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

BatchArgs batch_args(const dllm_batch* b, const dllm_cache* c) {
  BatchArgs a;
  a.block_table = b->block_table;
  a.seq_len = b->seq_len;
  a.block_start = b->block_start;
  a.block_len = b->block_len;
  a.cu_block = b->cu_block;
  a.cu_seq = b->cu_seq;
  a.err = b->error_flag;
  a.batch = b->batch;
  a.max_pages = b->max_pages_per_seq;
  a.num_pages = c->num_pages;
  a.max_block_len = b->max_block_len;
  a.max_seq_len = b->max_seq_len;
  a.total_block_rows = b->total_block_rows;
  a.total_seq_rows = b->total_seq_rows;
  return a;
}

float softmax_scale(const dllm_layer_desc* d) {
  return d->softmax_scale > 0.f ? d->softmax_scale : static_cast<float>(1.0 / sqrt(static_cast<double>(d->head_dim)));
}

AttnArgs attn_args(const dllm_layer_desc* d, const dllm_batch* b, const dllm_cache* c) {
  AttnArgs a;
  a.bt = batch_args(b, c);
  a.q_block = nullptr;
  a.k_pool = c->k_pool;
  a.v_pool = c->v_pool;
  a.q_pool = c->q_pool;
  a.m_pool = c->m_pool;
  a.l_pool = c->l_pool;
  a.o_pool = c->o_pool;
  a.o_full = nullptr;
  a.lse = nullptr;
  a.n_heads = d->n_heads;
  a.head_dim = d->head_dim;
  a.scale_log2 = softmax_scale(d) * 1.4426950408889634f;
  a.m_pre = nullptr;
  a.l_pre = nullptr;
  a.o_pre = nullptr;
  a.prev_start = nullptr;
  return a;
}

AttnPlan plan_of(const dllm_layer_desc* d, const dllm_batch* b, bool block, bool merge) {
  return attn_plan(b->batch, d->n_heads, d->head_dim, b->max_seq_len, b->max_block_len, b->total_seq_rows,
                   b->total_block_rows, device_sms(), block, merge);
}



QkvArgs qkv_args(const dllm_layer_desc* d, const dllm_batch* b, const dllm_cache* c, const float* rope,
                 int32_t rope_max_pos, int mode, int n_tok) {
  QkvArgs a;
  a.bt = batch_args(b, c);
  a.k_pool = c->k_pool;
  a.v_pool = c->v_pool;
  a.q_pool = c->q_pool;
  a.q_block = nullptr;
  a.rope = rope;
  a.rope_max_pos = rope_max_pos;
  a.n_heads = d->n_heads;
  a.head_dim = d->head_dim;
  a.d_model = d->d_model;
  a.n_tok = n_tok;
  a.mode = mode;
  a.x = nullptr;
  a.gain = nullptr;
  a.rms_eps = d->rms_eps;
  a.xhat = nullptr;
  a.inv = nullptr;
  a.norm_ctr = nullptr;
  a.partials = nullptr;
  a.counters = nullptr;
  a.max_contrib = 0;
  return a;
}

// Point the projection at its workspace: the counters (RMSNorm row claims,
// then the stream-K tile arrivals), the per-row RMSNorm scales, the x^ rows,
// and (stream-K) the fp32 partial tiles.
void bind_workspace(QkvArgs* a, const QkvPlan& plan, void* ws) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  a->norm_ctr = reinterpret_cast<int32_t*>(base);
  a->inv = reinterpret_cast<float2*>(base + plan.inv_offset);
  a->xhat = base + plan.xhat_offset;
  if (!plan.streamk) return;
  a->counters = reinterpret_cast<int32_t*>(base) + kQkvNormCounters;
  a->partials = reinterpret_cast<float*>(base + plan.part_offset);
  a->max_contrib = plan.max_contrib;
}

dllm_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DLLM_OK : DLLM_ERR_CUDA; }

#define DLLM_TRY(expr)                     \
  do {                                     \
    const dllm_status s_ = (expr);         \
    if (s_ != DLLM_OK) return s_;          \
  } while (0)

#define DLLM_CUDA_TRY(expr)                \
  do {                                     \
    const cudaError_t e_ = (expr);         \
    if (e_ != cudaSuccess) return DLLM_ERR_CUDA; \
  } while (0)

}  // namespace

extern "C" {

dllm_status dllm_workspace_size(const dllm_layer_desc* desc, const dllm_batch* batch, int32_t op, size_t* bytes) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  if (bytes == nullptr) return DLLM_ERR_INVALID_ARGUMENT;
  switch (op) {
    case DLLM_OP_CACHE_BUILD:
      *bytes = batch->batch > 0 && batch->total_seq_rows > 0
                   ? qkv_plan(batch->total_seq_rows, desc->d_model, desc->n_heads, desc->head_dim, device_sms())
                         .total_bytes
                   : 0;
      return DLLM_OK;
    case DLLM_OP_BLOCK_QKV_ROPE_WRITE:
      *bytes = batch->batch > 0 && batch->total_block_rows > 0
                   ? qkv_plan(batch->total_block_rows, desc->d_model, desc->n_heads, desc->head_dim, device_sms())
                         .total_bytes
                   : 0;
      return DLLM_OK;
    case DLLM_OP_BLOCK_ATTENTION:
      *bytes = batch->batch > 0 && batch->total_block_rows > 0 ? plan_of(desc, batch, true, false).total_bytes : 0;
      return DLLM_OK;
    case DLLM_OP_STEP_ATTENTION:
      *bytes = batch->batch > 0 && batch->total_block_rows > 0 ? plan_of(desc, batch, true, true).total_bytes : 0;
      return DLLM_OK;
    case DLLM_OP_STATE_MERGE:
      *bytes = 0;
      return DLLM_OK;
    case DLLM_OP_CACHE_ADVANCE:  // `batch` is the decoded blocks': the projection of their rows
      *bytes = batch->batch > 0 && batch->total_block_rows > 0
                   ? qkv_plan(batch->total_block_rows, desc->d_model, desc->n_heads, desc->head_dim, device_sms())
                         .total_bytes
                   : 0;
      return DLLM_OK;
    default:
      return DLLM_ERR_INVALID_ARGUMENT;
  }
}

dllm_status dllm_qkv_weight_packed_bytes(const dllm_layer_desc* desc, size_t* bytes) {
  if (bytes == nullptr) return DLLM_ERR_INVALID_ARGUMENT;
  DLLM_TRY(check_desc(desc));
  *bytes = qkv_packed_bytes(desc->d_model, desc->n_heads, desc->head_dim);
  return DLLM_OK;
}

dllm_status dllm_qkv_weight_pack(const dllm_layer_desc* desc, const void* w_qkv, void* w_packed, void* stream) {
  DLLM_TRY(check_desc(desc));
  if (!aligned(w_qkv, 16) || !aligned(w_packed, 16))
    return DLLM_ERR_INVALID_ARGUMENT;
  const size_t in_bytes = static_cast<size_t>(3) * desc->n_heads * desc->head_dim * desc->d_model * 2;
  const size_t out_bytes = qkv_packed_bytes(desc->d_model, desc->n_heads, desc->head_dim);
  const uintptr_t a = reinterpret_cast<uintptr_t>(w_qkv), b = reinterpret_cast<uintptr_t>(w_packed);
  if (a < b + out_bytes && b < a + in_bytes) return DLLM_ERR_INVALID_ARGUMENT;  // overlapping
  DLLM_CUDA_TRY(launch_qkv_pack(w_qkv, w_packed, 3 * desc->n_heads * desc->head_dim, desc->d_model,
                                static_cast<cudaStream_t>(stream)));
  return DLLM_OK;
}

dllm_status dllm_rope_table_build(const dllm_layer_desc* desc, int32_t max_pos, float* rope_table, void* stream) {
  DLLM_TRY(check_desc(desc));
  if (max_pos < 1 || !aligned(rope_table, 8)) return DLLM_ERR_INVALID_ARGUMENT;
  return cuda_status(launch_rope_table(rope_table, max_pos, desc->head_dim, static_cast<double>(desc->rope_theta),
                                       static_cast<cudaStream_t>(stream)));
}

dllm_status dllm_cache_build(const dllm_layer_desc* desc, const dllm_batch* batch, const void* x_full,
                             const void* rms_gain, const void* w_packed, const float* rope_table, int32_t rope_max_pos,
                             const dllm_cache* cache, void* ws, size_t ws_bytes, void* stream) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  if (batch->batch == 0 || batch->total_seq_rows == 0) return DLLM_OK;
  DLLM_TRY(check_cache(cache, desc, true, true));
  const int pre = pre_pools(cache);
  if (pre < 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned(x_full, 16) || !aligned(rms_gain, 16) || !aligned(w_packed, 16) || !aligned(rope_table, 8))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (rope_max_pos < batch->max_seq_len) return DLLM_ERR_INVALID_ARGUMENT;
  size_t need = 0;
  DLLM_TRY(dllm_workspace_size(desc, batch, DLLM_OP_CACHE_BUILD, &need));
  if (ws_bytes < need) return DLLM_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 256)) return DLLM_ERR_INVALID_ARGUMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  const BatchArgs bt = batch_args(batch, cache);
  const QkvPlan plan = qkv_plan(batch->total_seq_rows, desc->d_model, desc->n_heads, desc->head_dim, device_sms());
  QkvArgs qa = qkv_args(desc, batch, cache, rope_table, rope_max_pos, kModeBoundary, batch->total_seq_rows);
  qa.x = x_full;
  qa.gain = rms_gain;
  bind_workspace(&qa, plan, ws);
  DLLM_CUDA_TRY(launch_zero_tails(bt, cache->k_pool, cache->v_pool, cache->q_pool, desc->n_heads, desc->head_dim, s));
  DLLM_CUDA_TRY(launch_qkv_gemm(w_packed, qa, plan, s));
  AttnArgs aa = attn_args(desc, batch, cache);
  if (pre) {
    aa.m_pre = cache->m_pre;
    aa.l_pre = cache->l_pre;
    aa.o_pre = cache->o_pre;
  }
  DLLM_CUDA_TRY(launch_rows_attention(aa, pre ? kRowsStatePre : kRowsState, device_sms(), s));
  return DLLM_OK;
}

dllm_status dllm_cache_advance(const dllm_layer_desc* desc, const dllm_batch* batch, const dllm_batch* decoded,
                               const void* x_decoded, const void* rms_gain, const void* w_packed,
                               const float* rope_table, int32_t rope_max_pos, const dllm_cache* cache, void* ws,
                               size_t ws_bytes, void* stream) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  DLLM_TRY(check_batch(decoded));
  // the decoded blocks describe the same sequences, through the same metadata
  if (decoded->batch != batch->batch || decoded->block_table != batch->block_table ||
      decoded->seq_len != batch->seq_len || decoded->cu_seq != batch->cu_seq ||
      decoded->max_pages_per_seq != batch->max_pages_per_seq || decoded->total_seq_rows != batch->total_seq_rows ||
      decoded->max_seq_len != batch->max_seq_len)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (batch->batch == 0 || batch->total_seq_rows == 0) return DLLM_OK;
  DLLM_TRY(check_cache(cache, desc, true, true));
  if (pre_pools(cache) != 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned(x_decoded, 16) || !aligned(rms_gain, 16) || !aligned(w_packed, 16) || !aligned(rope_table, 8))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (rope_max_pos < batch->max_seq_len) return DLLM_ERR_INVALID_ARGUMENT;
  size_t need = 0;
  DLLM_TRY(dllm_workspace_size(desc, decoded, DLLM_OP_CACHE_ADVANCE, &need));
  if (ws_bytes < need) return DLLM_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && !aligned(ws, 256)) return DLLM_ERR_INVALID_ARGUMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  // the decoded rows: q, k, v into the pools
  if (decoded->total_block_rows > 0) {
    const QkvPlan plan =
        qkv_plan(decoded->total_block_rows, desc->d_model, desc->n_heads, desc->head_dim, device_sms());
    QkvArgs qa = qkv_args(desc, decoded, cache, rope_table, rope_max_pos, kModeRows, decoded->total_block_rows);
    qa.x = x_decoded;
    qa.gain = rms_gain;
    bind_workspace(&qa, plan, ws);
    DLLM_CUDA_TRY(launch_qkv_gemm(w_packed, qa, plan, s));
  }
  // the prefix state extended (rows kept) or rebuilt (decoded rows), then the state over U
  AttnArgs aa = attn_args(desc, batch, cache);
  aa.m_pre = cache->m_pre;
  aa.l_pre = cache->l_pre;
  aa.o_pre = cache->o_pre;
  aa.prev_start = decoded->block_start;
  DLLM_CUDA_TRY(launch_rows_attention(aa, kRowsAdvOld, device_sms(), s));
  DLLM_CUDA_TRY(launch_rows_attention(aa, kRowsAdvNew, device_sms(), s));
  return DLLM_OK;
}

dllm_status dllm_block_qkv_rope_write(const dllm_layer_desc* desc, const dllm_batch* batch, const void* x_block,
                                      const void* rms_gain, const void* w_packed, const float* rope_table,
                                      int32_t rope_max_pos, const dllm_cache* cache, void* q_block, void* ws,
                                      size_t ws_bytes, void* stream) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  if (batch->batch == 0 || batch->total_block_rows == 0) return DLLM_OK;
  DLLM_TRY(check_cache(cache, desc, false, false));
  if (!aligned(x_block, 16) || !aligned(rms_gain, 16) || !aligned(w_packed, 16) || !aligned(rope_table, 8) ||
      !aligned(q_block, 16))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (rope_max_pos < batch->max_seq_len) return DLLM_ERR_INVALID_ARGUMENT;
  size_t need = 0;
  DLLM_TRY(dllm_workspace_size(desc, batch, DLLM_OP_BLOCK_QKV_ROPE_WRITE, &need));
  if (ws_bytes < need) return DLLM_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 256)) return DLLM_ERR_INVALID_ARGUMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  const QkvPlan plan = qkv_plan(batch->total_block_rows, desc->d_model, desc->n_heads, desc->head_dim, device_sms());
  QkvArgs qa = qkv_args(desc, batch, cache, rope_table, rope_max_pos, kModeBlock, batch->total_block_rows);
  qa.q_block = q_block;
  qa.x = x_block;
  qa.gain = rms_gain;
  bind_workspace(&qa, plan, ws);
  DLLM_CUDA_TRY(launch_qkv_gemm(w_packed, qa, plan, s));
  return DLLM_OK;
}

namespace {
// The common part of the three attention calls: validate, bind the workspace, launch.
dllm_status attention_call(const dllm_layer_desc* desc, const dllm_batch* batch, const void* q_block,
                           const dllm_cache* cache, void* o_full, float* lse, void* ws, size_t ws_bytes, void* stream,
                           bool block, bool merge) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  if (batch->batch == 0 || batch->total_seq_rows == 0) return DLLM_OK;
  if (block && batch->total_block_rows == 0) block = false;
  if (!block && !merge) return DLLM_OK;
  // Blocks of at most one page run on the fused streaming kernel; longer blocks (the
  // prefix-only cache mode, where the block is everything after the prefix) on the
  // 128-row query-tile kernel, one launch per part.
  const bool wide = batch->max_block_len > kPage;
  if (!wide && !attn_batch_supported(batch->batch)) return DLLM_ERR_UNSUPPORTED;
  DLLM_TRY(check_cache(cache, desc, merge, merge));
  if (block && !aligned(q_block, 16)) return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned(o_full, 16)) return DLLM_ERR_INVALID_ARGUMENT;
  if (lse != nullptr && !aligned(lse, 4)) return DLLM_ERR_INVALID_ARGUMENT;
  const AttnPlan plan = plan_of(desc, batch, block, merge);
  if (ws_bytes < plan.total_bytes) return DLLM_ERR_WORKSPACE_TOO_SMALL;
  if (plan.total_bytes > 0 && !aligned(ws, 256)) return DLLM_ERR_INVALID_ARGUMENT;
  AttnArgs aa = attn_args(desc, batch, cache);
  aa.q_block = q_block;
  aa.o_full = o_full;
  aa.lse = lse;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (wide) {
    if (block) DLLM_CUDA_TRY(launch_rows_attention(aa, kRowsBlock, device_sms(), s));
    if (merge) DLLM_CUDA_TRY(launch_rows_attention(aa, kRowsMerge, device_sms(), s));
    return DLLM_OK;
  }
  DLLM_CUDA_TRY(launch_step_attention(aa, plan, s));
  return DLLM_OK;
}
}  // namespace

dllm_status dllm_block_attention(const dllm_layer_desc* desc, const dllm_batch* batch, const void* q_block,
                                 const dllm_cache* cache, void* o_full, float* lse, void* ws, size_t ws_bytes,
                                 void* stream) {
  return attention_call(desc, batch, q_block, cache, o_full, lse, ws, ws_bytes, stream, true, false);
}

dllm_status dllm_state_merge(const dllm_layer_desc* desc, const dllm_batch* batch, const dllm_cache* cache,
                             void* o_full, float* lse, void* ws, size_t ws_bytes, void* stream) {
  return attention_call(desc, batch, nullptr, cache, o_full, lse, ws, ws_bytes, stream, false, true);
}

dllm_status dllm_step_attention(const dllm_layer_desc* desc, const dllm_batch* batch, const void* q_block,
                                const dllm_cache* cache, void* o_full, float* lse, void* ws, size_t ws_bytes,
                                void* stream) {
  return attention_call(desc, batch, q_block, cache, o_full, lse, ws, ws_bytes, stream, true, true);
}

dllm_status dllm_lm_head_workspace_size(const dllm_layer_desc* desc, const dllm_batch* batch, int32_t vocab,
                                        size_t* bytes) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  if (bytes == nullptr || vocab < 1) return DLLM_ERR_INVALID_ARGUMENT;
  *bytes = batch->batch > 0 && batch->total_block_rows > 0
               ? lm_head_workspace_bytes(batch->total_block_rows, desc->d_model, vocab)
               : 0;
  return DLLM_OK;
}

dllm_status dllm_block_lm_head(const dllm_layer_desc* desc, const dllm_batch* batch, int32_t vocab,
                               const void* h_full, const void* final_gain, const void* w_lm, void* logits,
                               float* lse, int32_t* argmax, float* p_max, void* ws, size_t ws_bytes, void* stream) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  if (vocab < 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (desc->d_model % 128 != 0 || vocab % 8 != 0) return DLLM_ERR_UNSUPPORTED;
  if (batch->batch == 0 || batch->total_block_rows == 0) return DLLM_OK;
  if (!aligned(h_full, 16) || !aligned(final_gain, 16) || !aligned(w_lm, 16) || !aligned(lse, 4) ||
      !aligned(argmax, 4) || !aligned(p_max, 4))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (logits != nullptr && !aligned(logits, 16)) return DLLM_ERR_INVALID_ARGUMENT;
  size_t need = 0;
  DLLM_TRY(dllm_lm_head_workspace_size(desc, batch, vocab, &need));
  if (ws_bytes < need) return DLLM_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 256)) return DLLM_ERR_INVALID_ARGUMENT;
  LmArgs a;
  dllm_cache none = {};
  none.num_pages = 1;
  a.bt = batch_args(batch, &none);
  a.h = h_full;
  a.gain = final_gain;
  a.logits = logits;
  a.lse = lse;
  a.argmax = argmax;
  a.p_max = p_max;
  a.n_rows = batch->total_block_rows;
  a.d_model = desc->d_model;
  a.vocab = vocab;
  a.rms_eps = desc->rms_eps;
  lm_bind_workspace(&a, ws);
  DLLM_CUDA_TRY(launch_lm_head(w_lm, a, device_sms(), static_cast<cudaStream_t>(stream)));
  return DLLM_OK;
}

dllm_status dllm_ffn_workspace_size(const dllm_layer_desc* desc, const dllm_batch* batch, int32_t d_ff,
                                    size_t* bytes) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  if (bytes == nullptr || d_ff < 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (desc->d_model % 128 != 0 || d_ff % 128 != 0) return DLLM_ERR_UNSUPPORTED;
  *bytes = batch->batch > 0 && batch->total_block_rows > 0
               ? ffn_workspace_bytes(batch->total_block_rows, desc->d_model, desc->n_heads * desc->head_dim, d_ff,
                                     device_sms())
               : 0;
  return DLLM_OK;
}

dllm_status dllm_block_ffn(const dllm_layer_desc* desc, const dllm_batch* batch, int32_t d_ff, const void* o_full,
                           const void* x_block, const void* w_o, const void* ffn_gain, const void* w_gate_up,
                           const float* w_gate_up_scale, const void* w_down, const float* w_down_scale,
                           void* y_block, void* ws, size_t ws_bytes, void* stream) {
  size_t need = 0;
  DLLM_TRY(dllm_ffn_workspace_size(desc, batch, d_ff, &need));
  if (batch->batch == 0 || batch->total_block_rows == 0) return DLLM_OK;
  if (!aligned(o_full, 16) || !aligned(x_block, 16) || !aligned(w_o, 16) || !aligned(ffn_gain, 16) ||
      !aligned(w_gate_up, 16) || !aligned(w_gate_up_scale, 4) || !aligned(w_down, 16) || !aligned(w_down_scale, 4) ||
      !aligned(y_block, 16))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return DLLM_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 256)) return DLLM_ERR_INVALID_ARGUMENT;
  FfnArgs a = {};
  dllm_cache none = {};
  none.num_pages = 1;
  a.bt = batch_args(batch, &none);
  a.o_full = o_full;
  a.x_block = x_block;
  a.gain2 = ffn_gain;
  a.y = y_block;
  a.n_rows = batch->total_block_rows;
  a.d_model = desc->d_model;
  a.hd = desc->n_heads * desc->head_dim;
  a.d_ff = d_ff;
  a.rms_eps = desc->rms_eps;
  FfnWeights w;
  w.w_o = w_o;
  w.w_gu = w_gate_up;
  w.gu_scale = w_gate_up_scale;
  w.w_down = w_down;
  w.down_scale = w_down_scale;
  DLLM_CUDA_TRY(launch_ffn(a, w, ws, device_sms(), static_cast<cudaStream_t>(stream)));
  return DLLM_OK;
}

namespace {
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

dllm_status check_kv8(const dllm_kv8_cache* c, const dllm_layer_desc* d) {
  if (c == nullptr || c->num_pages < 1 || c->n_kv_heads < 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (d->n_heads % c->n_kv_heads != 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (static_cast<int64_t>(c->num_pages) * c->n_kv_heads * kPage > kMaxRows) return DLLM_ERR_UNSUPPORTED;
  if (!aligned(c->k_pool, 16) || !aligned(c->v_pool, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return DLLM_ERR_INVALID_ARGUMENT;
  return DLLM_OK;
}

Kv8Pools kv8_pools(const dllm_kv8_cache* c) {
  Kv8Pools p;
  p.k = static_cast<uint8_t*>(c->k_pool);
  p.v = static_cast<uint8_t*>(c->v_pool);
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.n_kv_heads = c->n_kv_heads;
  return p;
}

BatchArgs kv8_batch(const dllm_batch* b, int32_t num_pages) {
  dllm_cache pages = {};
  pages.num_pages = num_pages;
  return batch_args(b, &pages);
}

bool rows_ok(const void* p, int64_t row, int64_t head) {
  return aligned(p, 16) && row >= 0 && head >= 0 && row % 8 == 0 && head % 8 == 0;
}
}  // namespace

dllm_status dllm_batch_plan(const dllm_batch* batch, const int32_t* pages_held, int32_t* pages_held_out,
                            int32_t* block_table, int32_t* cu_block, int32_t* cu_seq, const dllm_page_ring* ring,
                            int32_t* row_slot, int32_t* row_seq, int32_t* row_pos, void* stream) {
  if (batch == nullptr || ring == nullptr || batch->batch < 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (batch->batch > 65535) return DLLM_ERR_UNSUPPORTED;
  if (!aligned(cu_block, 4) || !aligned(cu_seq, 4) || !aligned(ring->pages, 4) || !aligned(ring->state, 4) ||
      !aligned(ring->state_out, 4) || ring->num_pages < 1)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (ring->num_pages > kMaxRows / kPage) return DLLM_ERR_UNSUPPORTED;  // slots are int32
  if (overlap(ring->state, 8, ring->state_out, 8)) return DLLM_ERR_INVALID_ARGUMENT;
  if (batch->error_flag != nullptr && !aligned(batch->error_flag, 4)) return DLLM_ERR_INVALID_ARGUMENT;
  if (batch->total_block_rows < 0 || batch->total_seq_rows < 0) return DLLM_ERR_INVALID_ARGUMENT;
  for (const int32_t* p : {row_slot, row_seq, row_pos})
    if (p != nullptr && !aligned(p, 16)) return DLLM_ERR_INVALID_ARGUMENT;
  if (batch->batch > 0) {
    if (!aligned(batch->seq_len, 4) || !aligned(batch->block_start, 4) || !aligned(batch->block_len, 4) ||
        !aligned(pages_held, 4) || !aligned(pages_held_out, 4) || !aligned(block_table, 4))
      return DLLM_ERR_INVALID_ARGUMENT;
    const size_t n = static_cast<size_t>(batch->batch) * 4;
    if (overlap(pages_held, n, pages_held_out, n)) return DLLM_ERR_INVALID_ARGUMENT;
    if (batch->max_pages_per_seq < 1 || batch->max_seq_len < 1) return DLLM_ERR_INVALID_ARGUMENT;
    if (static_cast<int64_t>(batch->max_pages_per_seq) * kPage < batch->max_seq_len) return DLLM_ERR_INVALID_ARGUMENT;
    if (batch->max_seq_len > 65535 * kPage) return DLLM_ERR_UNSUPPORTED;
  }
  PlanArgs a;
  a.seq_len = batch->seq_len;
  a.block_start = batch->block_start;
  a.block_len = batch->block_len;
  a.held = pages_held;
  a.held_out = pages_held_out;
  a.table = block_table;
  a.cu_block = cu_block;
  a.cu_seq = cu_seq;
  a.ring = ring->pages;
  a.state = ring->state;
  a.state_out = ring->state_out;
  a.row_slot = row_slot;
  a.row_seq = row_seq;
  a.row_pos = row_pos;
  a.err = batch->error_flag;
  a.batch = batch->batch;
  a.max_pages = batch->max_pages_per_seq;
  a.num_pages = ring->num_pages;
  a.max_seq_len = batch->max_seq_len;
  a.cap_rows = batch->total_block_rows;
  a.cap_seq = batch->total_seq_rows;
  return cuda_status(launch_batch_plan(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

dllm_status dllm_kv8_write(const dllm_layer_desc* desc, const dllm_batch* batch, const void* k_rows,
                           int64_t k_row_stride, int64_t k_head_stride, const void* v_rows, int64_t v_row_stride,
                           int64_t v_head_stride, const dllm_kv8_cache* kv8, void* stream) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  if (batch->batch == 0 || batch->total_block_rows == 0) return DLLM_OK;
  DLLM_TRY(check_kv8(kv8, desc));
  if (!rows_ok(k_rows, k_row_stride, k_head_stride) || !rows_ok(v_rows, v_row_stride, v_head_stride))
    return DLLM_ERR_INVALID_ARGUMENT;
  Kv8WriteArgs a = {};
  a.bt = kv8_batch(batch, kv8->num_pages);
  a.kv = kv8_pools(kv8);
  a.k_src = k_rows;
  a.v_src = v_rows;
  a.k_row = k_row_stride;
  a.k_head = k_head_stride;
  a.v_row = v_row_stride;
  a.v_head = v_head_stride;
  a.head_dim = desc->head_dim;
  return cuda_status(launch_kv8_write(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

dllm_status dllm_kv8_write_pool(const dllm_layer_desc* desc, const dllm_batch* batch, const dllm_cache* cache,
                                const dllm_kv8_cache* kv8, void* stream) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  if (batch->batch == 0 || batch->total_block_rows == 0) return DLLM_OK;
  DLLM_TRY(check_cache(cache, desc, false, false));
  DLLM_TRY(check_kv8(kv8, desc));
  if (kv8->n_kv_heads != desc->n_heads) return DLLM_ERR_INVALID_ARGUMENT;
  Kv8WriteArgs a = {};
  a.bt = kv8_batch(batch, cache->num_pages < kv8->num_pages ? cache->num_pages : kv8->num_pages);
  a.kv = kv8_pools(kv8);
  a.k_src = cache->k_pool;
  a.v_src = cache->v_pool;
  a.head_dim = desc->head_dim;
  a.from_pool = true;
  return cuda_status(launch_kv8_write(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

dllm_status dllm_kv8_attention_workspace_size(const dllm_layer_desc* desc, const dllm_batch* batch,
                                              const dllm_kv8_cache* kv8, size_t* bytes) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  DLLM_TRY(check_kv8(kv8, desc));
  if (bytes == nullptr) return DLLM_ERR_INVALID_ARGUMENT;
  // rows that share a key head, and units of a sequence, are counted in 32 bits
  if (static_cast<int64_t>(batch->max_block_len) * desc->n_heads > kMaxRows) return DLLM_ERR_UNSUPPORTED;
  *bytes = batch->batch > 0 && batch->total_block_rows > 0
               ? kv8_attention_workspace_bytes(batch->max_block_len, desc->n_heads, kv8->n_kv_heads, desc->head_dim,
                                               device_sms())
               : 0;
  return DLLM_OK;
}

dllm_status dllm_kv8_attention(const dllm_layer_desc* desc, const dllm_batch* batch, const void* q,
                               int64_t q_row_stride, const dllm_kv8_cache* kv8, void* o, int32_t o_rows, float* lse,
                               void* ws, size_t ws_bytes, void* stream) {
  DLLM_TRY(check_desc(desc));
  DLLM_TRY(check_batch(batch));
  if (o_rows != DLLM_ROWS_BLOCK && o_rows != DLLM_ROWS_FULL) return DLLM_ERR_INVALID_ARGUMENT;
  if (batch->batch == 0 || batch->total_block_rows == 0) return DLLM_OK;
  size_t need = 0;
  DLLM_TRY(dllm_kv8_attention_workspace_size(desc, batch, kv8, &need));
  if (!aligned(q, 16) || q_row_stride % 8 != 0 || q_row_stride < static_cast<int64_t>(desc->n_heads) * desc->head_dim)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned(o, 16) || (lse != nullptr && !aligned(lse, 4))) return DLLM_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return DLLM_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 256)) return DLLM_ERR_INVALID_ARGUMENT;
  Kv8AttnArgs a = {};
  a.bt = kv8_batch(batch, kv8->num_pages);
  a.kv = kv8_pools(kv8);
  a.q = q;
  a.q_row = q_row_stride;
  a.o = o;
  a.lse = lse;
  a.full_rows = o_rows == DLLM_ROWS_FULL ? 1 : 0;
  a.n_heads = desc->n_heads;
  a.head_dim = desc->head_dim;
  a.scale_log2 = softmax_scale(desc) * 1.4426950408889634f;
  a.ws = ws;
  return cuda_status(launch_kv8_attention(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

namespace {
// Elements that rows and heads take up: heads of `len` at rs and hs elements (bf16), from p on.
struct Extent {
  const void* p;
  int64_t rows, rs, heads, hs, len;
  int64_t width() const { return (heads - 1) * hs + len; }              // of a row
  int64_t bytes() const { return ((rows - 1) * rs + width()) * 2; }
};

// Whether two sets of rows may share an element: no where their extents lie apart, where they are columns of
// the same wider rows that lie apart, or heads side by side at the same strides; yes otherwise.
bool may_overlap(const Extent& a, const Extent& b) {
  if (a.rows == 0 || b.rows == 0 || a.heads == 0 || b.heads == 0) return false;
  if (!overlap(a.p, a.bytes(), b.p, b.bytes())) return false;
  const int64_t bytes = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  if (bytes % 2 != 0) return true;
  // a's and b's pieces repeat every `step`: apart iff b's begins behind a's and ends before a's next
  auto apart = [&](int64_t step, int64_t len_a, int64_t len_b) {
    if (step <= 0) return false;
    const int64_t d = ((bytes / 2) % step + step) % step;
    return d >= len_a && d + len_b <= step;
  };
  if (a.rs == b.rs && apart(a.rs, a.width(), b.width())) return false;
  if (a.hs == b.hs && a.rs == b.rs && a.heads > 1 && b.heads > 1 && a.hs > 0 && a.rs % a.hs == 0 &&
      apart(a.hs, a.len, b.len))
    return false;
  return true;
}

dllm_status check_linear(const dllm_linear_layer* l, int32_t rows) {
  if (l == nullptr || rows < 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (l->in_features < 1 || l->out_features < 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (l->act < DLLM_ACT_NONE || l->act > DLLM_ACT_GELU_TANH) return DLLM_ERR_INVALID_ARGUMENT;
  if (l->gated != 0 && l->gated != 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (!(l->rms_eps >= 0.f) || !isfinite(l->rms_eps)) return DLLM_ERR_INVALID_ARGUMENT;
  if (l->in_features % 8 != 0) return DLLM_ERR_UNSUPPORTED;
  // tiles of 128 x 16 and coordinates are counted in 32 bits
  if (l->in_features > kMaxRows - 64 || l->out_features > (kMaxRows - 256) / 2 || rows > kMaxRows - 256)
    return DLLM_ERR_UNSUPPORTED;
  const int64_t wide = static_cast<int64_t>(l->out_features) * (l->gated ? 2 : 1);
  if (((wide + 127) / 128) * ((rows + int64_t{15}) / 16) > kMaxRows / 2) return DLLM_ERR_UNSUPPORTED;
  return DLLM_OK;
}

size_t linear_xhat_bytes(const dllm_linear_layer* l, int32_t rows) {
  return (static_cast<size_t>(rows) * l->in_features * 2 + 255) & ~static_cast<size_t>(255);
}
}  // namespace

dllm_status dllm_linear_workspace_size(const dllm_linear_layer* layer, int32_t rows, int32_t normed, size_t* bytes) {
  DLLM_TRY(check_linear(layer, rows));
  if (bytes == nullptr) return DLLM_ERR_INVALID_ARGUMENT;
  *bytes = normed ? linear_xhat_bytes(layer, rows) : 0;
  return DLLM_OK;
}

dllm_status dllm_linear(const dllm_linear_layer* layer, int32_t rows, const void* x, int64_t x_stride,
                        const void* rms_gain, const void* w, const void* bias, const void* residual,
                        int64_t residual_stride, void* y, int64_t y_stride, int32_t* error_flag, void* ws,
                        size_t ws_bytes, void* stream) {
  DLLM_TRY(check_linear(layer, rows));
  if (rows == 0) return DLLM_OK;
  const int64_t k = layer->in_features, n = layer->out_features, wide = layer->gated ? 2 * n : n;
  if (!aligned(x, 16) || x_stride % 8 != 0 || x_stride < k || !aligned(w, 16)) return DLLM_ERR_INVALID_ARGUMENT;
  if (x_stride > (int64_t{1} << 38)) return DLLM_ERR_UNSUPPORTED;  // a tensor map's strides are below 2^40 bytes
  if (rms_gain != nullptr && !aligned(rms_gain, 16)) return DLLM_ERR_INVALID_ARGUMENT;
  if (bias != nullptr && !aligned(bias, 2)) return DLLM_ERR_INVALID_ARGUMENT;
  if (residual != nullptr && (!aligned(residual, 2) || residual_stride < n)) return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned(y, 2) || y_stride < n) return DLLM_ERR_INVALID_ARGUMENT;
  if (error_flag != nullptr && !aligned(error_flag, 4)) return DLLM_ERR_INVALID_ARGUMENT;
  const Extent ye = {y, rows, y_stride, 1, 0, n};
  if (may_overlap(ye, {x, rows, x_stride, 1, 0, k}) || may_overlap(ye, {w, 1, 0, 1, 0, wide * k}) ||
      (rms_gain != nullptr && may_overlap(ye, {rms_gain, 1, 0, 1, 0, k})) ||
      (bias != nullptr && may_overlap(ye, {bias, 1, 0, 1, 0, wide})))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (residual != nullptr && !(residual == y && (residual_stride == y_stride || rows == 1)) &&
      may_overlap(ye, {residual, rows, residual_stride, 1, 0, n}))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (rms_gain != nullptr) {
    const size_t need = linear_xhat_bytes(layer, rows);
    if (ws_bytes < need) return DLLM_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(ws, 256)) return DLLM_ERR_INVALID_ARGUMENT;
    const Extent we = {ws, 1, 0, 1, 0, rows * k};
    if (may_overlap(we, ye) || may_overlap(we, {x, rows, x_stride, 1, 0, k}) || may_overlap(we, {w, 1, 0, 1, 0, wide * k}) ||
        may_overlap(we, {rms_gain, 1, 0, 1, 0, k}) || (bias != nullptr && may_overlap(we, {bias, 1, 0, 1, 0, wide})) ||
        (residual != nullptr && may_overlap(we, {residual, rows, residual_stride, 1, 0, n})))
      return DLLM_ERR_INVALID_ARGUMENT;
  }
  LinearArgs a = {};
  a.x = x;
  a.x_stride = x_stride;
  a.gain = rms_gain;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.r_stride = residual_stride;
  a.y = y;
  a.y_stride = y_stride;
  a.xhat = ws;
  a.err = error_flag;
  a.rows = rows;
  a.k = layer->in_features;
  a.n = layer->out_features;
  a.wide = static_cast<int32_t>(wide);
  a.act = layer->act;
  a.gated = layer->gated != 0;
  a.rms_eps = layer->rms_eps;
  return cuda_status(launch_linear(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

namespace {
Extent in_extent(const dllm_head_rows* h, int32_t rows, int32_t d) {
  return {h->in, rows, h->in_row_stride, h->n_heads, h->in_head_stride, d};
}
Extent out_extent(const dllm_head_rows* h, int32_t rows, int32_t d) {
  return {h->out, rows, h->out_row_stride, h->n_heads, h->out_head_stride, d};
}

dllm_status check_head_rows(const dllm_head_rows* h, int32_t rows, int32_t d) {
  if (h->n_heads < 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (static_cast<int64_t>(h->n_heads) * d > 65535 * 128) return DLLM_ERR_UNSUPPORTED;  // (as check_desc)
  if (!rows_ok(h->in, h->in_row_stride, h->in_head_stride) || !rows_ok(h->out, h->out_row_stride, h->out_head_stride))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (h->gain != nullptr && !aligned(h->gain, 16)) return DLLM_ERR_INVALID_ARGUMENT;
  if (h->in_row_stride > (int64_t{1} << 31) || h->in_head_stride > (int64_t{1} << 31) ||
      h->out_row_stride > (int64_t{1} << 31) || h->out_head_stride > (int64_t{1} << 31))
    return DLLM_ERR_UNSUPPORTED;  // offsets in 64 bits
  // the outputs' heads lie apart: heads within rows, or rows within heads
  const int64_t rs = h->out_row_stride, hs = h->out_head_stride;
  const bool heads_in_rows = (h->n_heads == 1 || hs >= d) && (rows <= 1 || rs >= (h->n_heads - 1) * hs + d);
  const bool rows_in_heads = (rows <= 1 || rs >= d) && (h->n_heads == 1 || hs >= (rows - 1) * rs + d);
  if (!heads_in_rows && !rows_in_heads) return DLLM_ERR_INVALID_ARGUMENT;
  const bool same = h->in == h->out && (rows <= 1 || h->in_row_stride == rs) &&
                    (h->n_heads == 1 || h->in_head_stride == hs);
  if (!same && may_overlap(out_extent(h, rows, d), in_extent(h, rows, d))) return DLLM_ERR_INVALID_ARGUMENT;
  return DLLM_OK;
}

HeadRows head_rows(const dllm_head_rows* h) {
  HeadRows r;
  r.in = h->in;
  r.in_row = h->in_row_stride;
  r.in_head = h->in_head_stride;
  r.out = h->out;
  r.out_row = h->out_row_stride;
  r.out_head = h->out_head_stride;
  r.gain = h->gain;
  r.n_heads = h->n_heads;
  return r;
}

// Whether rows of `len` elements of `size` bytes, `stride` elements apart from p on, share a byte with q's.
bool rows_hold(const void* p, int64_t rows, int64_t stride, int64_t len, int64_t size, const void* q, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
  if (y < x) return x - y < bytes;
  const int64_t first = static_cast<int64_t>((y - x) / size);  // elements behind p
  if (first >= (rows - 1) * stride + len) return false;
  const int64_t in_row = static_cast<int64_t>((y - x) % (stride * size));
  return in_row < len * size || in_row + bytes > static_cast<uint64_t>(stride * size);
}
}  // namespace

dllm_status dllm_head_norm_rope(const dllm_layer_desc* desc, int32_t rows, const int32_t* row_pos,
                                const dllm_head_rows* queries, const dllm_head_rows* keys, const float* rope_table,
                                int32_t rope_max_pos, int32_t rotary_dim, int32_t pairs, int32_t* error_flag,
                                void* stream) {
  DLLM_TRY(check_desc(desc));
  if (rows < 0 || queries == nullptr || rope_max_pos < 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (pairs != DLLM_ROPE_HALVES && pairs != DLLM_ROPE_NEIGHBOURS) return DLLM_ERR_INVALID_ARGUMENT;
  if ((rotary_dim != 64 && rotary_dim != 128) || rotary_dim > desc->head_dim) return DLLM_ERR_UNSUPPORTED;
  if (rows > kMaxRows - 256) return DLLM_ERR_UNSUPPORTED;  // counted in 32 bits, up to the end of a CTA's
  if (rows == 0) return DLLM_OK;
  const int32_t d = desc->head_dim;
  if (!aligned(row_pos, 4) || !aligned(rope_table, 16)) return DLLM_ERR_INVALID_ARGUMENT;
  if (error_flag != nullptr && !aligned(error_flag, 4)) return DLLM_ERR_INVALID_ARGUMENT;
  if (queries->n_heads != desc->n_heads) return DLLM_ERR_INVALID_ARGUMENT;
  DLLM_TRY(check_head_rows(queries, rows, d));
  const Extent pos = {row_pos, 1, 0, 1, 0, 2 * int64_t{rows}};
  const Extent table = {rope_table, 1, 0, 1, 0, 2 * int64_t{rope_max_pos} * rotary_dim};
  for (const dllm_head_rows* h : {queries, keys}) {
    if (h == nullptr) continue;
    if (h == keys) DLLM_TRY(check_head_rows(keys, rows, d));
    const Extent out = out_extent(h, rows, d);
    if (may_overlap(out, pos) || may_overlap(out, table)) return DLLM_ERR_INVALID_ARGUMENT;
    for (const dllm_head_rows* g : {queries, keys})
      if (g != nullptr && g->gain != nullptr && may_overlap(out, {g->gain, 1, 0, 1, 0, d}))
        return DLLM_ERR_INVALID_ARGUMENT;
  }
  if (keys != nullptr) {
    const Extent qi = in_extent(queries, rows, d), qo = out_extent(queries, rows, d);
    const Extent ki = in_extent(keys, rows, d), ko = out_extent(keys, rows, d);
    if (may_overlap(qo, ki) || may_overlap(qo, ko) || may_overlap(ko, qi)) return DLLM_ERR_INVALID_ARGUMENT;
  }
  HeadRopeArgs a = {};
  a.q = head_rows(queries);
  if (keys != nullptr) a.k = head_rows(keys);
  a.row_pos = row_pos;
  a.table = rope_table;
  a.err = error_flag;
  a.rows = rows;
  a.head_dim = d;
  a.max_pos = rope_max_pos;
  a.rotary_dim = rotary_dim;
  a.neighbours = pairs == DLLM_ROPE_NEIGHBOURS;
  a.eps = desc->rms_eps;
  return cuda_status(launch_head_rope(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

dllm_status dllm_token_scores(int32_t rows, int32_t vocab, const void* logits, int32_t logits_type, int64_t row_stride,
                              float scale, const int32_t* tokens, float* logp, float* lse, float* entropy,
                              int32_t top_k, int32_t* top_ids, float* top_logp, int32_t* error_flag, void* stream) {
  if (rows < 0 || vocab < 1 || top_k < 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (logits_type != DLLM_TYPE_BF16 && logits_type != DLLM_TYPE_FP32) return DLLM_ERR_INVALID_ARGUMENT;
  if (!(scale > 0.f) || !isfinite(scale)) return DLLM_ERR_INVALID_ARGUMENT;
  if (top_k > kMaxTop || vocab > (1 << 30) || rows > kMaxRows - 256) return DLLM_ERR_UNSUPPORTED;
  if (rows == 0) return DLLM_OK;
  const int size = logits_type == DLLM_TYPE_BF16 ? 2 : 4;
  if (!aligned(logits, size) || row_stride < vocab) return DLLM_ERR_INVALID_ARGUMENT;
  if (row_stride > (int64_t{1} << 31)) return DLLM_ERR_UNSUPPORTED;  // offsets in 64 bits
  if ((tokens == nullptr) != (logp == nullptr)) return DLLM_ERR_INVALID_ARGUMENT;
  for (const void* p : {static_cast<const void*>(tokens), static_cast<const void*>(logp), static_cast<const void*>(lse),
                        static_cast<const void*>(entropy), static_cast<const void*>(error_flag)})
    if (p != nullptr && !aligned(p, 4)) return DLLM_ERR_INVALID_ARGUMENT;
  if (top_k > 0 && (!aligned(top_ids, 4) || !aligned(top_logp, 4))) return DLLM_ERR_INVALID_ARGUMENT;
  // what is written lies apart from all else
  const size_t n = static_cast<size_t>(rows) * 4;
  const struct {
    const void* p;
    size_t bytes;
  } parts[] = {{logp, n}, {lse, n}, {entropy, n}, {top_k > 0 ? top_ids : nullptr, n * top_k},
               {top_k > 0 ? top_logp : nullptr, n * top_k}, {error_flag, 4}, {tokens, n}};
  for (int i = 0; i < 6; ++i) {
    if (parts[i].p == nullptr) continue;
    if (rows_hold(logits, rows, row_stride, vocab, size, parts[i].p, parts[i].bytes)) return DLLM_ERR_INVALID_ARGUMENT;
    for (int j = i + 1; j < 7; ++j)
      if (parts[j].p != nullptr && overlap(parts[i].p, parts[i].bytes, parts[j].p, parts[j].bytes))
        return DLLM_ERR_INVALID_ARGUMENT;
  }
  ScoreArgs a = {};
  a.logits = logits;
  a.stride = row_stride;
  a.tokens = tokens;
  a.logp = logp;
  a.lse = lse;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  a.err = error_flag;
  a.rows = rows;
  a.vocab = vocab;
  a.top = top_k;
  a.scale = scale;
  a.fp32 = logits_type == DLLM_TYPE_FP32;
  return cuda_status(launch_token_scores(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

const char* dllm_status_string(dllm_status status) {
  switch (status) {
    case DLLM_OK:
      return "ok";
    case DLLM_ERR_INVALID_ARGUMENT:
      return "invalid argument";
    case DLLM_ERR_UNSUPPORTED:
      return "unsupported shape or configuration";
    case DLLM_ERR_WORKSPACE_TOO_SMALL:
      return "workspace too small";
    case DLLM_ERR_CUDA:
      return "CUDA error";
    case DLLM_ERR_TIMEOUT:
      return "device wait timed out";
  }
  return "unknown status";
}

}  // extern "C"
