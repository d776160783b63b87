// linear.cu — products with a weight: y = act(x^ W^T + b) + r, also of gate and up units
// side by side, on tcgen05 (sm_103a).
//
//  * linear_norm_kernel  x^ = RMSNorm(x), correctly rounded to bf16, one CTA a row (only
//    where the call has a gain).
//  * linear_kernel       128 rows of W are the tensor core's M, up to 256 rows of x its N.
//    Warp 0 streams K in boxes of 64 through a ring, warp 1 issues the MMAs into TMEM, warps
//    2-5 turn the finished accumulators into y (a thread: one row of W; a warp's 32
//    neighbouring columns of y are one 64-byte run).
#include <math.h>

#include "layer_ops.cuh"
#include "norm.cuh"
#include "sm103.cuh"
#include "tmap.cuh"

namespace dllm {
namespace {

// ------------------------------------------------------------ RMSNorm
constexpr int kNormThreads = 256;

// x (s_hi + s_lo) g for 8 elements, correctly rounded to bf16.  t = x g is exact, t s_hi + t s_lo = p + e with |e| up to
// a step of p (half of one from p's rounding, half from s_lo); a second sum leaves |e| at most half a step, so that p alone
// decides unless it lies on a bf16 midpoint, where the sign of e does.
__device__ __forceinline__ uint4 normed8(const uint4& u, const uint4& gu, float s_hi, float s_lo) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w}, gw[4] = {gu.x, gu.y, gu.z, gu.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t half[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float xf = __uint_as_float(h ? (w[i] & 0xFFFF0000u) : (w[i] << 16));
      const float gv = __uint_as_float(h ? (gw[i] & 0xFFFF0000u) : (gw[i] << 16));
      const float t = __fmul_rn(xf, gv);
      const float p0 = __fmul_rn(t, s_hi);
      const float e0 = __fmaf_rn(t, s_lo, __fmaf_rn(t, s_hi, -p0));
      const float p = __fadd_rn(p0, e0), e = __fsub_rn(e0, __fsub_rn(p, p0));
      const uint32_t bits = __float_as_uint(p);
      const uint32_t rn = __bfloat16_as_ushort(__float2bfloat16_rn(p));
      const bool tie = (bits & 0xFFFFu) == 0x8000u && e != 0.f;
      const uint32_t away = ((e > 0.f) == (p > 0.f)) ? 1u : 0u;
      half[h] = tie ? (bits >> 16) + away : rn;
    }
    o[i] = (half[0] & 0xFFFFu) | (half[1] << 16);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kNormThreads) linear_norm_kernel(const LinearArgs a) {
  __shared__ float2 part[kNormThreads / 32];
  __shared__ float2 scale;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nvec = a.k / 8;
  griddep_wait();
  griddep_launch_dependents();
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + blockIdx.x * a.x_stride);
  uint4* out = static_cast<uint4*>(a.xhat) + static_cast<size_t>(blockIdx.x) * nvec;
  const uint4* g = static_cast<const uint4*>(a.gain);
  float hi = 0.f, lo = 0.f;
  for (int v = threadIdx.x; v < nvec; v += kNormThreads) sumsq_pair_add(__ldg(x + v), hi, lo);
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    const float oh = __shfl_xor_sync(0xffffffffu, hi, o), ol = __shfl_xor_sync(0xffffffffu, lo, o);
    pair_add(hi, lo, oh, ol);
  }
  if (lane == 0) part[warp] = make_float2(hi, lo);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kNormThreads / 32; ++w) pair_add(hi, lo, part[w].x, part[w].y);
    two_sum(hi, lo, hi, lo);
    float2 s;
    rsqrt_pair(hi, lo, a.k, a.rms_eps, s.x, s.y);
    scale = s;
  }
  __syncthreads();
  const float2 s = scale;
  for (int v = threadIdx.x; v < nvec; v += kNormThreads) out[v] = normed8(__ldg(x + v), __ldg(g + v), s.x, s.y);
}

// ------------------------------------------------------------ the epilogue's arithmetic
template <int ACT>
__device__ __forceinline__ float activate(float t) {
  if (ACT == kActSilu) return t / (1.f + expf(-t));
  if (ACT == kActGelu) return 0.5f * t * (1.f + erff(t * 0.70710678118654752f));
  if (ACT == kActGeluTanh) return 0.5f * t * (1.f + tanhf(0.79788456080286536f * (t + 0.044715f * t * t * t)));
  return t;
}

__device__ __forceinline__ float bf16_at(const void* p, int64_t i) {
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// ------------------------------------------------------------ the product
constexpr int kThreads = 192;
constexpr int kBK = 64;
constexpr int kTW = 128;                 // rows of W to a tile (tcgen05 M)
constexpr int kABytes = kTW * kBK * 2;
constexpr int kMaxStages = 12;
constexpr int kRingBytes = 200 * 1024;

struct LinearTiles {
  int bn;      // rows of x to a tile (tcgen05 N): a multiple of 16
  int stages;  // of the ring
  int boxes;   // of K
  uint32_t cols;  // TMEM columns
};

template <int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const LinearArgs a,
                  const LinearTiles t) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  __shared__ uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], done_bar;
  __shared__ uint32_t tmem_base_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stage_bytes = kABytes + t.bn * kBK * 2;
  const int w0 = blockIdx.x * kTW, x0 = blockIdx.y * t.bn;

  if (threadIdx.x == 0) {
    for (int s = 0; s < t.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&done_bar, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) tmem_alloc(&tmem_base_sh, t.cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  if (warp == 0) {
    if (lane == 0) {
      griddep_wait();
      griddep_launch_dependents();
      bool ok = true;
      int kb = 0;
      for (; kb < t.boxes && ok; ++kb) {
        const int s = kb % t.stages;
        if (kb >= t.stages && !mbar_wait(&empty_bar[s], (kb / t.stages - 1) & 1)) {
          ok = false;
          break;
        }
        uint8_t* st = smem + s * stage_bytes;
        mbar_arrive_expect_tx(&full_bar[s], stage_bytes);
        tma_load_2d(st, &tm_w, &full_bar[s], kb * kBK, w0);  // rows past W's, and x's, read 0
        tma_load_2d(st + kABytes, &tm_x, &full_bar[s], kb * kBK, x0);
      }
      for (int i = kb > t.stages ? kb - t.stages : 0; i < kb; ++i)  // every load has landed before the CTA ends
        ok = mbar_wait(&full_bar[i % t.stages], (i / t.stages) & 1) && ok;
      if (!ok) report_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = umma_idesc_bf16(kTW, t.bn);
      bool ok = true;
      for (int kb = 0; kb < t.boxes && ok; ++kb) {
        const int s = kb % t.stages;
        ok = mbar_wait(&full_bar[s], (kb / t.stages) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + s * stage_bytes), sb = sa + kABytes;
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          umma_bf16(tmem, umma_desc_sw128(sa + kk * 32), umma_desc_sw128(sb + kk * 32), idesc,
                    (kb > 0 || kk > 0) ? 1u : 0u);
        if (kb + t.stages < t.boxes) umma_commit(&empty_bar[s]);  // the last ones no load waits for
      }
      umma_commit(&done_bar);
      if (!ok) report_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    const int quad = warp & 3;
    const int wr = w0 + quad * 32 + lane;  // this thread's row of W
    const bool row_there = wr < a.wide;
    griddep_wait();  // the residual, and y behind whoever reads it
    const float b = row_there && a.bias != nullptr ? bf16_at(a.bias, wr) : 0.f;
    if (!mbar_wait(&done_bar, 0)) report_error(a.err, kErrTimeout);
    tc_fence_after();
    const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int rows = min(t.bn, a.rows - x0);
    const int n = GATED ? wr >> 1 : wr;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y);
    for (int c0 = 0; c0 < rows; c0 += 16) {
      float v[16];
      tmem_ld_32x32b_x16(src + c0, v);
      if (GATED) {
        // the even lane has the gate of 16 rows, the odd one the up: each makes y of eight of them
        const bool up = lane & 1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float mine = (up ? v[8 + i] : v[i]) + b, give = (up ? v[i] : v[8 + i]) + b;
          const float other = __shfl_xor_sync(0xffffffffu, give, 1);
          const float g = up ? other : mine, u = up ? mine : other;
          const int c = c0 + (up ? 8 : 0) + i;
          if (row_there && c < rows) {
            float o = activate<ACT>(g) * u;
            if (a.residual != nullptr) o += bf16_at(a.residual, (x0 + c) * a.r_stride + n);
            y[(x0 + c) * a.y_stride + n] = __float2bfloat16_rn(o);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = c0 + i;
          if (row_there && c < rows) {
            float o = activate<ACT>(v[i] + b);
            if (a.residual != nullptr) o += bf16_at(a.residual, (x0 + c) * a.r_stride + n);
            y[(x0 + c) * a.y_stride + n] = __float2bfloat16_rn(o);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, t.cols);
  }
}

template <int ACT, bool GATED>
cudaError_t launch_product(const LinearArgs& a, cudaStream_t stream) {
  LinearTiles t;
  t.bn = a.rows >= 256 ? 256 : (a.rows + 15) / 16 * 16;
  t.boxes = (a.k + kBK - 1) / kBK;
  const int stage = kABytes + t.bn * kBK * 2;
  t.stages = kRingBytes / stage;
  t.stages = t.stages > kMaxStages ? kMaxStages : t.stages;
  t.stages = t.stages > t.boxes ? t.boxes : t.stages;
  t.cols = 32;
  while (t.cols < static_cast<uint32_t>(t.bn)) t.cols *= 2;
  CUtensorMap tm_w, tm_x;
  cudaError_t e = encode_rows_sw128(&tm_w, a.w, a.k, a.wide, a.k, kBK, kTW);
  if (e == cudaSuccess)
    e = a.gain != nullptr ? encode_rows_sw128(&tm_x, a.xhat, a.k, a.rows, a.k, kBK, t.bn)
                          : encode_rows_sw128(&tm_x, a.x, a.k, a.rows, a.x_stride, kBK, t.bn);
  if (e != cudaSuccess) return e;
  const int smem = t.stages * stage + 1024;
  e = cudaFuncSetAttribute(linear_kernel<ACT, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.wide + kTW - 1) / kTW, (a.rows + t.bn - 1) / t.bn);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_kernel<ACT, GATED>, tm_w, tm_x, a, t);
}

template <int ACT>
cudaError_t launch_act(const LinearArgs& a, cudaStream_t stream) {
  return a.gated ? launch_product<ACT, true>(a, stream) : launch_product<ACT, false>(a, stream);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  if (a.rows <= 0) return cudaSuccess;
  if (a.gain != nullptr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.rows);
    cfg.blockDim = dim3(kNormThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, linear_norm_kernel, a);
    if (e != cudaSuccess) return e;
  }
  switch (a.act) {
    case kActSilu:
      return launch_act<kActSilu>(a, stream);
    case kActGelu:
      return launch_act<kActGelu>(a, stream);
    case kActGeluTanh:
      return launch_act<kActGeluTanh>(a, stream);
    default:
      return launch_act<kActNone>(a, stream);
  }
}

}  // namespace dllm
