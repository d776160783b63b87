// head_rope.cu — the norm of each head of packed queries and keys and their rotation by
// position, in one pass (sm_103a):
//   u = x / sqrt(mean(x^2) + eps) * g,   (u_a, u_b) -> (u_a cos - u_b sin, u_a sin + u_b cos)
// in fp32, rounded to bf16 once.
//
// A head is d / 16 lanes with two 16-byte pieces each, chosen so that both elements of every
// pair lie with one lane: pieces l and l + rotary_dim / 16 where halves turn together, 2 l
// and 2 l + 1 where neighbours do (the lanes behind the rotated elements take theirs two by
// two).  So the only exchange is the sum of squares, over 8 (d = 128) or 4 lanes, and a warp
// instruction moves whole 128-byte runs of 4 or 8 heads.  A lane's eight pairs have the same
// numbers in every head: their cos and sin are loaded once for all heads of a row.
#include "layer_ops.cuh"
#include "sm103.cuh"

namespace dllm {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// A warp: one row's heads [first, first + kStep), [first + kStep, ...) of the queries, then of the keys.
template <int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kWarps * 32) head_rope_kernel(const HeadRopeArgs a) {
  constexpr int kLanes = D / 16;         // lanes of a head
  constexpr int kStep = 32 / kLanes;     // heads of a warp instruction
  const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (row >= a.rows) return;
  const int pos = __ldg(a.row_pos + row);
  if (pos < 0 || pos >= a.max_pos) {
    if (pos != -1 && lane == 0) report_error(a.err, kErrBadShape);
    return;
  }
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
  float cs[16];
  if (turns) {
    const float4* t = reinterpret_cast<const float4*>(a.table + (static_cast<size_t>(pos) * turned + l) * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(t + i);
      cs[4 * i] = f.x;
      cs[4 * i + 1] = f.y;
      cs[4 * i + 2] = f.z;
      cs[4 * i + 3] = f.w;
    }
  }
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const HeadRows& r = side ? a.k : a.q;
    const uint16_t* in = static_cast<const uint16_t*>(r.in) + row * r.in_row;
    uint16_t* out = static_cast<uint16_t*>(r.out) + row * r.out_row;
    uint4 g0 = {}, g1 = {};
    const bool norm = r.gain != nullptr;
    if (norm) {
      g0 = __ldg(static_cast<const uint4*>(r.gain) + p0);
      g1 = __ldg(static_cast<const uint4*>(r.gain) + p1);
    }
#pragma unroll 2
    for (int h = sub; h < r.n_heads + sub; h += kStep) {  // the same turns for every lane
      const bool there = h < r.n_heads;
      uint4 u0 = {}, u1 = {};
      if (there) {
        const uint4* src = reinterpret_cast<const uint4*>(in + h * r.in_head);
        u0 = src[p0];
        u1 = src[p1];
      }
      float x0[8], x1[8];
      unpack8(u0, x0);
      unpack8(u1, x1);
      if (norm) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], s));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float inv = rsqrtf(s * (1.f / D) + a.eps);
        float w0[8], w1[8];
        unpack8(g0, w0);
        unpack8(g1, w1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x0[i] = x0[i] * inv * w0[i];
          x1[i] = x1[i] * inv * w1[i];
        }
      }
      if (turns) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& p = NEIGHBOURS ? (i < 4 ? x0[2 * i] : x1[2 * i - 8]) : x0[i];
          float& q = NEIGHBOURS ? (i < 4 ? x0[2 * i + 1] : x1[2 * i - 7]) : x1[i];
          const float c = cs[2 * i], s = cs[2 * i + 1], u = p;
          p = u * c - q * s;
          q = u * s + q * c;
        }
      }
      if (there) {
        uint4* dst = reinterpret_cast<uint4*>(out + h * r.out_head);
        dst[p0] = pack8(x0);
        dst[p1] = pack8(x1);
      }
    }
  }
}

}  // namespace

cudaError_t launch_head_rope(const HeadRopeArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  if (a.rows <= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.rows + kWarps - 1) / kWarps);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.head_dim == 128)
    return a.neighbours ? cudaLaunchKernelEx(&cfg, head_rope_kernel<128, true>, a)
                        : cudaLaunchKernelEx(&cfg, head_rope_kernel<128, false>, a);
  return a.neighbours ? cudaLaunchKernelEx(&cfg, head_rope_kernel<64, true>, a)
                      : cudaLaunchKernelEx(&cfg, head_rope_kernel<64, false>, a);
}

}  // namespace dllm
