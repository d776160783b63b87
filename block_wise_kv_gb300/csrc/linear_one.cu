// linear_one.cu — the product with a weight of a single row, y = act(x^ W^T + b) + r (sm_103a).
//
// Nothing of W is used twice, so that there is nothing for tensor cores to gain, and their way
// in and out costs: K has to be cut over clusters for all SMs to read W, and the parts meet
// again.  Here a CTA takes an even share of W's rows, whole; a team of 32 to 1024 threads lies
// along K.  A thread keeps its one or two pieces of x^ in registers (normed there, while W is
// on its way) and streams its pieces of W past them, four pieces at work and four on their way,
// with two multiply-adds to an instruction.  A warp's lanes are added up by halves, so that
// kBatch rows cost little more shuffles than one; the warps' sums meet in shared memory and
// are added in the order of K.
//
// Bound by HBM: 4096 x 6144 9.3 us (floor 7.4; a library product 10.1), normed 10.4; 4096 x
// 2 x 12288 gated and normed 34 (29.7, 5.9 TB/s); small ones by their way through memory: 2.0.
#include "linear_math.cuh"

namespace dllm {
namespace {

constexpr int kRows = 128;  // rows of W to a CTA, at most
template <int P>
constexpr int kBatch = 4 / P;  // rows that a team takes at a time

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 u;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}

// The sums of v over a warp's lanes: of U values, lane (32 / U) i has that of v[i].
template <int U>
__device__ __forceinline__ float warp_sums(float (&v)[U], int lane) {
  int o = 16;
#pragma unroll
  for (int n = U / 2; n > 0; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

template <int T, int P, int ACT, bool GATED>
__global__ void __launch_bounds__(T, 1024 / T) linear_one_kernel(const LinearArgs a, int team) {
  constexpr int U = kBatch<P>, kWarps = T / 32;
  __shared__ float part[kWarps][kRows];  // [warp of a team][row of W]
  __shared__ float2 norm_part[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nvec = a.k / 8;
  const int teams = T / team, mine = threadIdx.x / team, l = threadIdx.x % team, w_in = warp % (team / 32);
  constexpr int kUnit = GATED ? 2 : 1;  // rows of W that stay together
  const int lo = kUnit * static_cast<int>(static_cast<int64_t>(a.n) * blockIdx.x / gridDim.x);
  const int hi = kUnit * static_cast<int>(static_cast<int64_t>(a.n) * (blockIdx.x + 1) / gridDim.x);
  const uint4* w = static_cast<const uint4*>(a.w);
  griddep_wait();
  griddep_launch_dependents();

  auto ask = [&](int r, uint4 (&q)[U][P]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = r + u * teams + mine;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int v = l + p * team;
        q[u][p] = row < hi && v < nvec ? ld_stream(w + static_cast<int64_t>(row) * nvec + v) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  uint4 x[P], qa[U][P], qb[U][P];
#pragma unroll
  for (int p = 0; p < P; ++p)
    x[p] = l + p * team < nvec ? __ldg(static_cast<const uint4*>(a.x) + l + p * team) : make_uint4(0u, 0u, 0u, 0u);
  const int batch = U * teams;
  ask(lo, qa);
  ask(lo + batch, qb);
  const int i_out = threadIdx.x, j = lo / kUnit + i_out;  // this thread's column of y
  const bool out = i_out < (hi - lo) / kUnit;
  float b0 = 0.f, b1 = 0.f, r0 = 0.f;
  if (out) {
    if (a.bias != nullptr) {
      b0 = bf16_at(a.bias, static_cast<int64_t>(kUnit) * j);
      if (GATED) b1 = bf16_at(a.bias, 2 * static_cast<int64_t>(j) + 1);
    }
    if (a.residual != nullptr) r0 = bf16_at(a.residual, j);
  }
  if (a.gain != nullptr) {
    uint4 g[P];
#pragma unroll
    for (int p = 0; p < P; ++p)
      g[p] = l + p * team < nvec ? __ldg(static_cast<const uint4*>(a.gain) + l + p * team) : make_uint4(0u, 0u, 0u, 0u);
    float2 hi2 = {0.f, 0.f}, lo2 = {0.f, 0.f};
#pragma unroll
    for (int p = 0; p < P; ++p) sumsq2_add(x[p], hi2, lo2);
    float sh, sl;
    sums_of(hi2, lo2, sh, sl);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float oh = __shfl_xor_sync(0xffffffffu, sh, o), ol = __shfl_xor_sync(0xffffffffu, sl, o);
      pair_add(sh, sl, oh, ol);
    }
    if (lane == 0) norm_part[warp] = make_float2(sh, sl);  // lane 0's sum is the warp's
    __syncthreads();
    sh = norm_part[0].x;  // the first team's: all have the same
    sl = norm_part[0].y;
    for (int i = 1; i < team / 32; ++i) pair_add(sh, sl, norm_part[i].x, norm_part[i].y);
    two_sum(sh, sl, sh, sl);
    float s_hi, s_lo;
    rsqrt_pair(sh, sl, a.k, a.rms_eps, s_hi, s_lo);
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = normed8(x[p], g[p], s_hi, s_lo);
  }

  auto use = [&](int r, const uint4 (&q)[U][P]) {
    float2 s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = make_float2(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t xw[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 xv = unpack2(xw[e]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t qw[4] = {q[u][p].x, q[u][p].y, q[u][p].z, q[u][p].w};
          s[u] = fma2(unpack2(qw[e]), xv, s[u]);
        }
      }
    }
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = s[u].x + s[u].y;
    const float sum = warp_sums<U>(v, lane);
    const int row = r + lane / (32 / U) * teams + mine;
    if (lane % (32 / U) == 0 && row < hi) part[w_in][row - lo] = sum;
  };
#pragma unroll 1
  for (int r = lo; r < hi; r += 2 * batch) {
    use(r, qa);
    ask(r + 2 * batch, qa);
    if (r + batch < hi) {
      use(r + batch, qb);
      ask(r + 3 * batch, qb);
    }
  }
  __syncthreads();
  if (!out) return;
  float t0 = 0.f, t1 = 0.f;
  for (int i = 0; i < team / 32; ++i) {
    t0 += part[i][kUnit * i_out];
    if (GATED) t1 += part[i][kUnit * i_out + 1];
  }
  const float o = GATED ? activate<ACT>(t0 + b0) * (t1 + b1) : activate<ACT>(t0 + b0);
  static_cast<__nv_bfloat16*>(a.y)[j] = __float2bfloat16_rn(o + r0);
}

template <int T, int P, int ACT, bool GATED>
cudaError_t launch_one(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  int team = 32;
  while (team * 8 * P < a.k) team *= 2;
  // A CTA to each SM as long as each has a batch of rows, more where each has four (512 x 12288: 5.2 us, 5.8 with four CTAs an
  // SM that have little more than one; 256 x 768 2.0, 2.4 with a CTA to each SM).
  const int batch = kBatch<P> * (T / team), batches = (a.wide + batch - 1) / batch, most = 1024 / T * num_sms;
  int ctas = batches < num_sms ? batches : batches / 4 < num_sms ? num_sms : batches / 4;
  ctas = ctas < most ? ctas : most;
  const int least = (a.wide + kRows - 1) / kRows + 1;
  ctas = ctas < least ? least : ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(T);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_one_kernel<T, P, ACT, GATED>, a, team);
}

// (1024 threads an SM hold any K's x^ as two pieces each and W's as eight: 4096 x 6144 on two CTAs of 512 threads, a piece
// each, 9.6 us, not 9.3; 12288 x 4096 with four pieces each, which spill, 24.)
template <int ACT, bool GATED>
cudaError_t launch_one_k(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  return a.k <= 2048   ? launch_one<256, 1, ACT, GATED>(a, num_sms, stream)
         : a.k <= 4096 ? launch_one<256, 2, ACT, GATED>(a, num_sms, stream)
         : a.k <= 8192 ? launch_one<512, 2, ACT, GATED>(a, num_sms, stream)
                       : launch_one<1024, 2, ACT, GATED>(a, num_sms, stream);
}

template <int ACT>
cudaError_t launch_one_act(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  return a.gated ? launch_one_k<ACT, true>(a, num_sms, stream) : launch_one_k<ACT, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_linear_one(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  switch (a.act) {
    case kActSilu:
      return launch_one_act<kActSilu>(a, num_sms, stream);
    case kActGelu:
      return launch_one_act<kActGelu>(a, num_sms, stream);
    case kActGeluTanh:
      return launch_one_act<kActGeluTanh>(a, num_sms, stream);
    default:
      return launch_one_act<kActNone>(a, num_sms, stream);
  }
}

}  // namespace dllm
