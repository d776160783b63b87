// linear_few.cu — the product with a weight of one or two rows, y = act(x^ W^T + b) + r (sm_103a).
//
// So little is done with W that there is nothing for tensor cores to gain, and their way in and
// out costs: K has to be cut over clusters for all SMs to read W, and the parts meet again.
// Here a CTA takes an even share of W's rows, whole; a team of 32 to 1024 threads lies along K.
// A thread keeps its one or two pieces of x^ in registers (normed there, while W is on its way)
// and streams its pieces of W past them, four at work and four on their way, with two
// multiply-adds to an instruction.  A warp's lanes are added up by halves, so that the sums of
// kBatch rows cost little more shuffles than one; the warps' sums meet in shared memory and
// are added in the order of K.
//
// Bound by HBM: one row 4096 x 6144 9.2 us (floor 7.4; a library product 10.1), normed 10.6;
// 4096 x 2 x 12288 gated and normed 34 (29.7: 5.9 TB/s); two rows 10.5, 12.5 and 36.  Small ones by
// their way through memory: 2.0.
#include "linear_math.cuh"

namespace dllm {
namespace {

template <int P>
constexpr int kBatch = 4 / P;   // rows of W that a team takes at a time, P pieces to a thread
constexpr int kMostRows = 128;  // rows of W to a CTA: a thread makes one value of y

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 u;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}

// The sums of N values v over a warp's lanes: lane (32 / N) i has that of v[i].
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
  int o = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

template <int T, int C, int R, int P, int ACT, bool GATED>
__global__ void __launch_bounds__(T, C) linear_few_kernel(const LinearArgs a, int team) {
  constexpr int U = kBatch<P>, kWarps = T / 32, N = U * R;
  __shared__ float part[kWarps][R][kMostRows];  // [warp of a team][row of x][row of W]
  __shared__ float2 norm_part[R][kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nvec = a.k / 8;
  const int teams = T / team, mine = threadIdx.x / team, l = threadIdx.x % team, w_in = warp % (team / 32);
  constexpr int kUnit = GATED ? 2 : 1;  // rows of W that stay together
  const int j0 = static_cast<int>(static_cast<int64_t>(a.n) * blockIdx.x / gridDim.x);
  const int cols = static_cast<int>(static_cast<int64_t>(a.n) * (blockIdx.x + 1) / gridDim.x) - j0;  // of y
  const int lo = kUnit * j0, hi = lo + kUnit * cols, batch = U * teams;
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
  uint4 x[R][P], qa[U][P], qb[U][P];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + i * a.x_stride);
#pragma unroll
    for (int p = 0; p < P; ++p)
      x[i][p] = (R == 1 || i < a.rows) && l + p * team < nvec ? __ldg(from + l + p * team) : make_uint4(0u, 0u, 0u, 0u);
  }
  ask(lo, qa);
  ask(lo + batch, qb);
  // this thread's value of y, in row m and column j0 + c
  const int m = R == 1 ? 0 : threadIdx.x / kMostRows, c = threadIdx.x - m * kMostRows;
  const bool out = m < a.rows && c < cols;
  float b0 = 0.f, b1 = 0.f, r0 = 0.f;
  if (out) {
    if (a.bias != nullptr) {
      b0 = bf16_at(a.bias, static_cast<int64_t>(kUnit) * (j0 + c));
      if (GATED) b1 = bf16_at(a.bias, 2 * static_cast<int64_t>(j0 + c) + 1);
    }
    if (a.residual != nullptr) r0 = bf16_at(a.residual, m * a.r_stride + j0 + c);
  }
  if (a.gain != nullptr) {
    uint4 g[P];
#pragma unroll
    for (int p = 0; p < P; ++p)
      g[p] = l + p * team < nvec ? __ldg(static_cast<const uint4*>(a.gain) + l + p * team) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float2 hi2 = {0.f, 0.f}, lo2 = {0.f, 0.f};
#pragma unroll
      for (int p = 0; p < P; ++p) sumsq2_add(x[i][p], hi2, lo2);
      float sh, sl;
      sums_of(hi2, lo2, sh, sl);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float oh = __shfl_xor_sync(0xffffffffu, sh, o), ol = __shfl_xor_sync(0xffffffffu, sl, o);
        pair_add(sh, sl, oh, ol);
      }
      if (lane == 0) norm_part[i][warp] = make_float2(sh, sl);  // lane 0's sum is the warp's
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float sh = norm_part[i][0].x, sl = norm_part[i][0].y;  // the first team's: all have the same
      for (int k = 1; k < team / 32; ++k) pair_add(sh, sl, norm_part[i][k].x, norm_part[i][k].y);
      two_sum(sh, sl, sh, sl);
      float s_hi, s_lo;
      rsqrt_pair(sh, sl, a.k, a.rms_eps, s_hi, s_lo);
#pragma unroll
      for (int p = 0; p < P; ++p) x[i][p] = normed8(x[i][p], g[p], s_hi, s_lo);
    }
  }

  auto use = [&](int r, const uint4 (&q)[U][P]) {
    float2 s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 xv[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const uint32_t xw[4] = {x[i][p].x, x[i][p].y, x[i][p].z, x[i][p].w};
          xv[i] = unpack2(xw[e]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t qw[4] = {q[u][p].x, q[u][p].y, q[u][p].z, q[u][p].w};
          const float2 wv = unpack2(qw[e]);
#pragma unroll
          for (int i = 0; i < R; ++i) s[i * U + u] = fma2(wv, xv[i], s[i * U + u]);
        }
      }
    }
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = s[i].x + s[i].y;
    const float sum = warp_sums<N>(v, lane);
    const int i = lane / (32 / N), row = r + i % U * teams + mine;
    if (lane % (32 / N) == 0 && row < hi) part[w_in][i / U][row - lo] = sum;
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
  float t0 = b0, t1 = b1;
  for (int i = 0; i < team / 32; ++i) {
    t0 += part[i][m][kUnit * c];
    if (GATED) t1 += part[i][m][kUnit * c + 1];
  }
  const float o = GATED ? activate<ACT>(t0) * t1 : activate<ACT>(t0);
  static_cast<__nv_bfloat16*>(a.y)[m * a.y_stride + j0 + c] = __float2bfloat16_rn(o + r0);
}

template <int T, int C, int R, int P, int ACT, bool GATED>
cudaError_t launch(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  int team = 32;
  while (team * 8 * P < a.k) team *= 2;
  // A CTA to each SM as long as each has a batch of rows, more where each has four (512 x 12288: 5.2 us, 5.8 with four CTAs an
  // SM that have little more than one; 256 x 768 2.0, 2.4 with a CTA to each SM).
  const int batch = kBatch<P> * (T / team), batches = (a.wide + batch - 1) / batch, most = C * num_sms;
  int ctas = batches < num_sms ? batches : batches / 4 < num_sms ? num_sms : batches / 4;
  ctas = ctas < most ? ctas : most;
  const int least = (a.wide + kMostRows - 1) / kMostRows + 1;
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
  return cudaLaunchKernelEx(&cfg, linear_few_kernel<T, C, R, P, ACT, GATED>, a, team);
}

// (One row: 1024 threads an SM hold any K's x^ as two pieces each and W's as eight, in 64 registers but for some 70 bytes a
// thread that spill, 24 to 48 with one piece: 4096 x 6144 on two CTAs of 512 threads, a piece each, 9.6 us, not 9.3;
// 12288 x 4096 with four pieces each, which spill more, 24 for 17.  Two rows: half the threads, with twice the registers and
// no spills.)
template <int ACT, bool GATED>
cudaError_t launch_k(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  if (a.rows == 2)
    return a.k <= 2048 ? launch<256, 2, 2, 1, ACT, GATED>(a, num_sms, stream)
                       : launch<256, 2, 2, 2, ACT, GATED>(a, num_sms, stream);
  return a.k <= 2048   ? launch<256, 4, 1, 1, ACT, GATED>(a, num_sms, stream)
         : a.k <= 4096 ? launch<256, 4, 1, 2, ACT, GATED>(a, num_sms, stream)
         : a.k <= 8192 ? launch<512, 2, 1, 2, ACT, GATED>(a, num_sms, stream)
                       : launch<1024, 1, 1, 2, ACT, GATED>(a, num_sms, stream);
}

template <int ACT>
cudaError_t launch_act(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  return a.gated ? launch_k<ACT, true>(a, num_sms, stream) : launch_k<ACT, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_linear_few(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  switch (a.act) {
    case kActSilu:
      return launch_act<kActSilu>(a, num_sms, stream);
    case kActGelu:
      return launch_act<kActGelu>(a, num_sms, stream);
    case kActGeluTanh:
      return launch_act<kActGeluTanh>(a, num_sms, stream);
    default:
      return launch_act<kActNone>(a, num_sms, stream);
  }
}

}  // namespace dllm
