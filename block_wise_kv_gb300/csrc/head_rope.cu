// head_rope.cu — the norm of each head of packed queries and keys and their rotation by
// position, in one pass (sm_103a):
//   u = x / sqrt(mean(x^2) + eps) * g,   (u_a, u_b) -> (u_a cos - u_b sin, u_a sin + u_b cos)
// in fp32, rounded to bf16 once.
//
// A head is d / 16 lanes with two 16-byte pieces each, chosen so that both elements of every
// pair lie with one lane: pieces l and l + rotary_dim / 16 where halves turn together, 2 l
// and 2 l + 1 where neighbours do (the lanes behind the rotated elements take theirs two by
// two).  So the only exchange is the sum of squares, over 8 (d = 128) or 4 lanes, and a warp
// instruction moves whole 128-byte runs of 4 or 8 heads: a step.  A warp takes some of a
// row's steps, three on their way in shared memory (a lane's own pieces, so that nothing waits
// for another lane) while one is worked on; its position, and behind that the cos and sin of
// each lane's eight pairs, the same in every head, come once.
//
// Bound by HBM where rows are many (20480 rows of 32 and 8 heads of 128: 65 us, 6.4 TB/s, a
// copy of as much 61; 76 with two steps on their way in registers, which left room for 20
// warps an SM and not 28, 82 with such warps that go on from row to row; 95 with four steps of
// a row to a warp and no loop), by the way to the position, the table and the row where they
// are few (64 rows: 2.1 us, a step to a warp; 5.7 with a row to a warp).
#include "layer_ops.cuh"
#include "pairs.cuh"
#include "sm103.cuh"

namespace dllm {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void unpack8(const uint4& u, float2 (&v)[4]) {
  v[0] = unpack2(u.x);
  v[1] = unpack2(u.y);
  v[2] = unpack2(u.z);
  v[3] = unpack2(u.w);
}

__device__ __forceinline__ uint4 pack8(const float2 (&v)[4]) {
  return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                    pack_bf16x2(v[3].x, v[3].y));
}

constexpr int kRing = 4;  // steps that a warp has on their way or at work

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Warp: row blockIdx.x kWarps + its number, steps [y per, (y + 1) per) with y = blockIdx.y, of the queries' and then the
// keys'.
template <int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kWarps * 32, 7) head_rope_kernel(const HeadRopeArgs a, int per) {
  constexpr int kLanes = D / 16;         // lanes of a head
  constexpr int kHeads = 32 / kLanes;    // heads of a step
  const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (row >= a.rows) return;
  const int pos = __ldg(a.row_pos + row);
  const int q_steps = (a.q.n_heads + kHeads - 1) / kHeads;
  const int first = blockIdx.y * per;
  const int end = min(first + per, q_steps + (a.k.n_heads + kHeads - 1) / kHeads);
  const int turned = a.rotary_dim / 16;  // lanes whose elements turn
  const bool turns = l < turned;
  int p0, p1;  // this lane's pieces of a head
  if (NEIGHBOURS) {
    p0 = 2 * l;
    p1 = p0 + 1;
  } else {
    p0 = turns ? l : 2 * l;  // behind the 2 turned pieces: 2 turned + 2 (l - turned)
    p1 = turns ? l + turned : p0 + 1;
  }
  const uint16_t* q_in = static_cast<const uint16_t*>(a.q.in) + row * a.q.in_row + sub * a.q.in_head;
  const uint16_t* k_in = static_cast<const uint16_t*>(a.k.in) + row * a.k.in_row + sub * a.k.in_head;
  __shared__ uint4 held[kWarps][kRing][2][32];  // a lane's pieces, which no other reads
  const uint4* const mine = &held[threadIdx.x >> 5][0][0][lane];
  auto ask = [&](int s, int place) {
    if (s < end) {
      const bool is_k = s >= q_steps;
      const int h0 = (is_k ? s - q_steps : s) * kHeads;
      if (h0 + sub < (is_k ? a.k.n_heads : a.q.n_heads)) {
        const uint4* src = reinterpret_cast<const uint4*>(is_k ? k_in + h0 * a.k.in_head : q_in + h0 * a.q.in_head);
        const uint32_t to = smem_u32(mine + place * 64);
        cp_async16(to, src + p0);
        cp_async16(to + 512, src + p1);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) ask(first + i, i);
  if (pos < 0 || pos >= a.max_pos) {
    if (pos != -1 && lane == 0) report_error(a.err, kErrBadShape);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  float2 cs[8];  // of the lane's pairs; halves: cos of two and sin of two in turn
  if (turns) {
    const float4* t = reinterpret_cast<const float4*>(a.table + (static_cast<size_t>(pos) * turned + l) * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(t + i);
      cs[2 * i] = NEIGHBOURS ? make_float2(f.x, f.y) : make_float2(f.x, f.z);
      cs[2 * i + 1] = NEIGHBOURS ? make_float2(f.z, f.w) : make_float2(f.y, f.w);
    }
  }
  uint16_t* q_out = static_cast<uint16_t*>(a.q.out) + row * a.q.out_row + sub * a.q.out_head;
  uint16_t* k_out = static_cast<uint16_t*>(a.k.out) + row * a.k.out_row + sub * a.k.out_head;
  uint4 g0 = {}, g1 = {};
  bool norm = false;
  int place = 0;
#pragma unroll 1
  for (int s = first; s < end; ++s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
    const uint4 u0 = mine[place * 64], u1 = mine[place * 64 + 32];  // (lanes without a head: whatever lies there, not stored)
    ask(s + kRing - 1, place == 0 ? kRing - 1 : place - 1);  // where the step before lay
    place = place + 1 == kRing ? 0 : place + 1;
    const bool is_k = s >= q_steps;
    if (s == first || s == q_steps) {  // the gains of this side
      const void* gain = is_k ? a.k.gain : a.q.gain;
      norm = gain != nullptr;
      if (norm) {
        g0 = __ldg(static_cast<const uint4*>(gain) + p0);
        g1 = __ldg(static_cast<const uint4*>(gain) + p1);
      }
    }
    float2 x0[4], x1[4];
    unpack8(u0, x0);
    unpack8(u1, x1);
    if (norm) {
      float2 sq = mul2(x0[0], x0[0]);
#pragma unroll
      for (int k = 1; k < 4; ++k) sq = fma2(x0[k], x0[k], sq);
#pragma unroll
      for (int k = 0; k < 4; ++k) sq = fma2(x1[k], x1[k], sq);
      float sum = sq.x + sq.y;
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float inv = rsqrtf(sum * (1.f / D) + a.eps);
      float2 w0[4], w1[4];
      unpack8(g0, w0);
      unpack8(g1, w1);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x0[k] = mul2(mul2(x0[k], {inv, inv}), w0[k]);
        x1[k] = mul2(mul2(x1[k], {inv, inv}), w1[k]);
      }
    }
    if (turns) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (NEIGHBOURS) {
          float2 &p = x0[k], &q = x1[k];
          p = make_float2(p.x * cs[k].x - p.y * cs[k].y, p.x * cs[k].y + p.y * cs[k].x);
          q = make_float2(q.x * cs[4 + k].x - q.y * cs[4 + k].y, q.x * cs[4 + k].y + q.y * cs[4 + k].x);
        } else {
          const float2 c = cs[2 * k], n = cs[2 * k + 1], u = x0[k], v = x1[k];
          const float2 w = mul2(v, n);
          x0[k] = fma2(u, c, make_float2(-w.x, -w.y));
          x1[k] = fma2(u, n, mul2(v, c));
        }
      }
    }
    const int h0 = (is_k ? s - q_steps : s) * kHeads;
    if (h0 + sub < (is_k ? a.k.n_heads : a.q.n_heads)) {
      uint4* dst = reinterpret_cast<uint4*>(is_k ? k_out + h0 * a.k.out_head : q_out + h0 * a.q.out_head);
      dst[p0] = pack8(x0);
      dst[p1] = pack8(x1);
    }
  }
}

template <int D, bool NEIGHBOURS>
cudaError_t launch(const HeadRopeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int kHeads = 512 / D;
  const int steps = (a.q.n_heads + kHeads - 1) / kHeads + (a.k.n_heads + kHeads - 1) / kHeads;
  // As many steps to a warp as leave every SM some twenty warps, the same for all.
  const int64_t most = static_cast<int64_t>(a.rows) * steps / (20 * num_sms);
  int per = most < 1 ? 1 : most > steps ? steps : static_cast<int>(most);
  const int parts = (steps + per - 1) / per;
  per = (steps + parts - 1) / parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.rows + kWarps - 1) / kWarps, parts);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, head_rope_kernel<D, NEIGHBOURS>, a, per);
}

}  // namespace

cudaError_t launch_head_rope(const HeadRopeArgs& a, int num_sms, cudaStream_t stream) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.head_dim == 128) return a.neighbours ? launch<128, true>(a, num_sms, stream) : launch<128, false>(a, num_sms, stream);
  return a.neighbours ? launch<64, true>(a, num_sms, stream) : launch<64, false>(a, num_sms, stream);
}

}  // namespace dllm
