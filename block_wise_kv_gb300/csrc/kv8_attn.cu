// kv8_attn.cu — attention of the block rows over the e4m3 paged cache (simple form:
// one warp per block row and query head, a lane per key for the scores, the online
// softmax over 32 keys at a time).
#include "attn_common.cuh"
#include "kv8.cuh"

namespace dllm {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float2 e4m3x2_f32(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv8_attn_kernel(const Kv8AttnArgs a) {
  __shared__ float qs[kWarps][D];
  const BatchArgs& bt = a.bt;
  const int b = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.n_heads / a.kv.n_kv_heads;
  griddep_wait();
  griddep_launch_dependents();
  const int n = bt.seq_len[b], s = bt.block_start[b], rows = bt.block_len[b], cub = bt.cu_block[b], cus = bt.cu_seq[b];
  if (rows == 0 || n == 0) return;
  if (n < 0 || n > bt.max_seq_len || rows < 0 || rows > bt.max_block_len || s < 0 || rows > n - s || cub < 0 ||
      rows > bt.total_block_rows - cub || (a.full_rows && (cus < 0 || n > bt.total_seq_rows - cus)) ||
      (n + kPage - 1) / kPage > bt.max_pages) {
    if (threadIdx.x == 0) report_error(bt.err, kErrBadShape);
    return;
  }
  constexpr int kE = D / 32;
  for (int r = warp; r < rows * G; r += kWarps) {
    const int i = r / G, head = h * G + r % G;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (cub + i) * a.q_row + head * D;
    __syncwarp();
    for (int c = lane; c < D; c += 32) qs[warp][c] = __bfloat162float(q[c]) * a.scale_log2;
    __syncwarp();
    float m = attn::neg_inf(), l = 0.f, o[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = 0.f;
    for (int k0 = 0; k0 < n; k0 += 32) {
      const int pg = attn::page_of(bt, b, k0 / kPage);
      const size_t slot = (static_cast<size_t>(pg) * a.kv.n_kv_heads + h) * kPage + k0 % kPage;
      const size_t sc = (static_cast<size_t>(pg) * a.kv.n_kv_heads + h) * kKv8Groups + (k0 % kPage + lane) / kKv8Group;
      const bool on = k0 + lane < n;
      float x = attn::neg_inf(), vs = 0.f;
      if (on) {
        x = 0.f;
        for (int c = 0; c < D; c += 2) {
          const float2 kv = e4m3x2_f32(*reinterpret_cast<const uint16_t*>(a.kv.k + (slot + lane) * D + c));
          x += kv.x * qs[warp][c] + kv.y * qs[warp][c + 1];
        }
        x *= a.kv.k_scale[sc];
        vs = a.kv.v_scale[sc];
      }
      float mx = x;
      for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float mn = fmaxf(m, mx), alpha = attn::fast_exp2(m - mn), p = on ? exp2f(x - mn) : 0.f;
      m = mn;
      float ps = p;
      for (int d = 16; d > 0; d >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, d);
      l = l * alpha + ps;
#pragma unroll
      for (int e = 0; e < kE; ++e) o[e] *= alpha;
      const int keys = min(32, n - k0);
      for (int j = 0; j < keys; ++j) {
        const float w = __shfl_sync(0xffffffffu, p * vs, j);
#pragma unroll
        for (int e = 0; e < kE; e += 2) {
          const float2 v = e4m3x2_f32(*reinterpret_cast<const uint16_t*>(a.kv.v + (slot + j) * D + lane * kE + e));
          o[e] += w * v.x;
          o[e + 1] += w * v.y;
        }
      }
    }
    const size_t row = a.full_rows ? cus + s + i : cub + i;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + (row * a.n_heads + head) * D;
#pragma unroll
    for (int e = 0; e < kE; ++e) out[lane * kE + e] = __float2bfloat16(o[e] / l);
    if (a.lse != nullptr && lane == 0) a.lse[row * a.n_heads + head] = (m + log2f(l)) * attn::kLn2;
  }
}

}  // namespace

size_t kv8_attention_workspace_bytes(int, int, int, int, int) { return 4096; }

cudaError_t launch_kv8_attention(const Kv8AttnArgs& a, int, cudaStream_t stream) {
  const dim3 grid(a.bt.batch, a.kv.n_kv_heads);
  if (a.head_dim == 128) return attn::launch_pdl(kv8_attn_kernel<128>, grid, kWarps * 32, 0, 0, stream, a);
  return attn::launch_pdl(kv8_attn_kernel<64>, grid, kWarps * 32, 0, 0, stream, a);
}

}  // namespace dllm
