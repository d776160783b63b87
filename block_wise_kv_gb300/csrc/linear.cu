// linear.cu — products with a weight: y = act(x^ W^T + b) + r, also of gate and up units
// side by side, on tcgen05 (sm_103a).
//
//  * linear_norm_kernel  x^ = RMSNorm(x), correctly rounded to bf16, one CTA a row (only
//    where the call has a gain).
//  * linear_rows_kernel  few rows: 128 rows of W are the tensor core's M, up to 256 rows of
//    x its N.  K is cut over the CTAs of a cluster, so that all SMs read W; the parts meet in
//    shared memory, each CTA adds up some of the columns in the order of K.  Warp 0 streams
//    boxes of 64 columns through a ring, warp 1 issues the MMAs into TMEM, warps 2-5 make y
//    (a thread: one row of W; a warp's 32 neighbouring columns of y are one 64-byte run).
//  * linear_tiles_kernel many rows: a pair of CTAs (cta_group::2) takes 256 rows of x by up
//    to 256 rows of W, each CTA half of either operand, and walks such tiles.  Two
//    accumulators in TMEM: warps 2-5 of each CTA make y of one tile (a thread: one row of x)
//    while the tensor cores work on the next, through a staging tile that makes whole runs
//    of the rows of y and of the residual.
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

// ------------------------------------------------------------ few rows
constexpr int kThreads = 192;
constexpr int kBK = 64;
constexpr int kTW = 128;                 // rows of W to a tile (tcgen05 M)
constexpr int kABytes = kTW * kBK * 2;
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;             // CTAs of a cluster

struct RowsPlan {
  int bn;         // rows of x to a tile (tcgen05 N): a multiple of 16
  int split;      // CTAs that share a tile's K
  int stages;     // of the ring
  int boxes;      // of K
  int per_rank;   // groups of 4 rows of x that each CTA of a cluster finishes
  uint32_t cols;  // TMEM columns
  int xt;         // tiles of x
};

__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x),
               "r"(y)
               : "memory");
}

// y of four rows of x (x0 + c ...) under this thread's row of W, whose sums are v.
template <int ACT, bool GATED>
__device__ __forceinline__ void finish4(const LinearArgs& a, const float (&v)[4], float b, int wr, int row, int lane) {
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y);
  if (GATED) {
    // the even lane has the gate of four rows, the odd one the up: each makes y of two of them
    const bool up = lane & 1;
    const int n = wr >> 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float mine = (up ? v[2 + i] : v[i]) + b, give = (up ? v[i] : v[2 + i]) + b;
      const float other = __shfl_xor_sync(0xffffffffu, give, 1);
      const float g = up ? other : mine, u = up ? mine : other;
      const int64_t r = row + (up ? 2 : 0) + i;
      if (wr < a.wide && r < a.rows) {
        float o = activate<ACT>(g) * u;
        if (a.residual != nullptr) o += bf16_at(a.residual, r * a.r_stride + n);
        y[r * a.y_stride + n] = __float2bfloat16_rn(o);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = row + i;
      if (wr < a.wide && r < a.rows) {
        float o = activate<ACT>(v[i] + b);
        if (a.residual != nullptr) o += bf16_at(a.residual, r * a.r_stride + wr);
        y[r * a.y_stride + wr] = __float2bfloat16_rn(o);
      }
    }
  }
}

template <int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    linear_rows_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                       const LinearArgs a, const RowsPlan t) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  __shared__ uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], done_bar;
  __shared__ uint32_t tmem_base_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stage_bytes = kABytes + t.bn * kBK * 2;
  const int rank = static_cast<int>(blockIdx.x) % t.split, tile = static_cast<int>(blockIdx.x) / t.split;
  const int w0 = tile / t.xt * kTW, x0 = tile % t.xt * t.bn;  // tiles that share rows of W side by side
  const int kb0 = static_cast<int>(static_cast<int64_t>(t.boxes) * rank / t.split);
  const int nb = static_cast<int>(static_cast<int64_t>(t.boxes) * (rank + 1) / t.split) - kb0;

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
  const int quad = warp & 3;
  const int wr = w0 + quad * 32 + lane;  // warps 2-5: this thread's row of W
  float b = 0.f;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      const int early = nb < t.stages ? nb : t.stages;
      // What stands in front may still be writing W, but where that is the norm kernel, which starts this one only
      // behind its own wait.  Elsewhere the first boxes of W go as far as L2.
      if (a.gain != nullptr) {
        for (int i = 0; i < early; ++i) {
          mbar_arrive_expect_tx(&full_bar[i], stage_bytes);
          tma_load_2d(smem + i * stage_bytes, &tm_w, &full_bar[i], (kb0 + i) * kBK, w0);
        }
      } else {
        for (int i = 0; i < early; ++i) tma_prefetch_2d(&tm_w, (kb0 + i) * kBK, w0);
      }
      griddep_wait();
      griddep_launch_dependents();
      int i = 0;
      for (; i < nb && ok; ++i) {
        const int s = i % t.stages;
        uint8_t* st = smem + s * stage_bytes;
        if (i >= t.stages && !mbar_wait(&empty_bar[s], (i / t.stages - 1) & 1)) {
          ok = false;
          break;
        }
        if (i >= early || a.gain == nullptr) {
          mbar_arrive_expect_tx(&full_bar[s], stage_bytes);
          tma_load_2d(st, &tm_w, &full_bar[s], (kb0 + i) * kBK, w0);  // rows past W's, and x's, read 0
        }
        tma_load_2d(st + kABytes, &tm_x, &full_bar[s], (kb0 + i) * kBK, x0);
      }
      for (int j = i > t.stages ? i - t.stages : 0; j < i; ++j)  // every load has landed before the ring ends
        ok = mbar_wait(&full_bar[j % t.stages], (j / t.stages) & 1) && ok;
      if (!ok) report_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = umma_idesc_bf16(kTW, t.bn);
      bool ok = true;
      for (int i = 0; i < nb; ++i) {
        const int s = i % t.stages;
        ok = mbar_wait(&full_bar[s], (i / t.stages) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + s * stage_bytes), sb = sa + kABytes;
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          umma_bf16(tmem, umma_desc_sw128(sa + kk * 32), umma_desc_sw128(sb + kk * 32), idesc,
                    (i > 0 || kk > 0) ? 1u : 0u);
        if (i + t.stages < nb) umma_commit(&empty_bar[s]);  // the last ones no load waits for
      }
      umma_commit(&done_bar);
      if (!ok) report_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    griddep_wait();  // bias, residual, and y behind whoever reads it
    b = wr < a.wide && a.bias != nullptr ? bf16_at(a.bias, wr) : 0.f;
    if (!mbar_wait(&done_bar, 0)) report_error(a.err, kErrTimeout);
    tc_fence_after();
  }
  const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  if (t.split == 1) {
    if (warp >= 2) {
      for (int c0 = 0; c0 < t.bn && x0 + c0 < a.rows; c0 += 16) {
        float v[16];
        tmem_ld_32x32b_x16(src + c0, v);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float w[4] = {v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
          finish4<ACT, GATED>(a, w, b, wr, x0 + c0 + 4 * g, lane);
        }
      }
    }
  } else {
    // The rings are done with on all sides; each CTA's sums of group g (four rows of x) go to the CTA that
    // finishes it: [CTA they come from][group][row of W], 16 bytes each.
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    const uint32_t mine = smem_u32(smem) + (quad * 32 + lane) * 16;
    if (warp >= 2) {
      for (int c0 = 0; c0 < t.bn; c0 += 16) {
        float v[16];
        tmem_ld_32x32b_x16(src + c0, v);
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
          const int g = c0 / 4 + g4, to = g / t.per_rank;
          st_shared_cluster_v4(mapa_shared(mine + (rank * t.per_rank + g - to * t.per_rank) * (kTW * 16), to),
                               make_float4(v[4 * g4], v[4 * g4 + 1], v[4 * g4 + 2], v[4 * g4 + 3]));
        }
      }
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    if (warp >= 2) {
      const float4* part = reinterpret_cast<const float4*>(smem) + quad * 32 + lane;
      for (int g = 0; g < t.per_rank; ++g) {
        const int c = (rank * t.per_rank + g) * 4;
        if (c >= t.bn || x0 + c >= a.rows) break;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < t.split; ++r) {
          const float4 p = part[(r * t.per_rank + g) * kTW];
          v[0] += p.x;
          v[1] += p.y;
          v[2] += p.z;
          v[3] += p.w;
        }
        finish4<ACT, GATED>(a, v, b, wr, x0 + c, lane);
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

// ------------------------------------------------------------ many rows
constexpr int kPairRows = 256;           // rows of x to a pair's tile
constexpr int kPairStages = 6;
constexpr int kHalfBytes = 128 * kBK * 2;  // a CTA's half of an operand's box, at most
constexpr int kPairStage = 2 * kHalfBytes;
constexpr int kStageCols = 64;           // columns of y in a staging tile: 128-byte rows
constexpr int kStageTile = 32 * kStageCols * 2;
constexpr int kPairSmem = kPairStages * kPairStage + 4 * 2 * kStageTile + 1024;

struct TilesPlan {
  int bn;      // rows of W to a tile: a multiple of 32, at most 256
  int boxes;   // of K
  int wt, xt;  // tiles of W, of x
  int pairs;   // CTA pairs
  bool y_vec, r_vec;  // rows of y, of the residual on 16-byte boundaries
};

__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void umma_bf16_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrive at the barrier at this place in both CTAs once all MMAs issued so far are done.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// As mbar_wait, behind arrivals from both CTAs.
__device__ __forceinline__ bool mbar_wait_pair(uint64_t* bar, uint32_t parity) {
  const bool ok = mbar_wait(bar, parity);
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
  return ok;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Columns [c0, c0 + kStageCols) of 32 rows of y or the residual, as one warp moves them to or from its staging
// tile (rows of 128 bytes, 16-byte pieces swizzled by the row).
__device__ __forceinline__ void residual_to_stage(const LinearArgs& a, bool vec, uint8_t* stage, int64_t row0, int c0,
                                                  int cols, int lane) {
  const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(a.residual);
  if (vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = i * 4 + lane / 8, piece = lane & 7, c = c0 + piece * 8;
      if (row0 + row >= a.rows || piece * 8 >= cols) continue;
      const __nv_bfloat16* p = r + (row0 + row) * a.r_stride + c;
      if (c + 8 <= a.n) {
        cp_async16(smem_u32(stage) + sw128_offset(row, piece), p);
      } else {
        for (int e = 0; c + e < a.n; ++e) reinterpret_cast<__nv_bfloat16*>(stage + sw128_offset(row, piece))[e] = p[e];
      }
    }
  } else {
    for (int row = 0; row < 32 && row0 + row < a.rows; ++row)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = h * 32 + lane, c = c0 + e;
        if (e < cols && c < a.n)
          reinterpret_cast<__nv_bfloat16*>(stage + sw128_offset(row, e >> 3))[e & 7] = r[(row0 + row) * a.r_stride + c];
      }
  }
  cp_async_commit();
}

__device__ __forceinline__ void stage_to_y(const LinearArgs& a, bool vec, const uint8_t* stage, int64_t row0, int c0,
                                           int cols, int lane) {
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y);
  if (vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = i * 4 + lane / 8, piece = lane & 7, c = c0 + piece * 8;
      if (row0 + row >= a.rows || piece * 8 >= cols) continue;
      __nv_bfloat16* p = y + (row0 + row) * a.y_stride + c;
      const uint4 u = *reinterpret_cast<const uint4*>(stage + sw128_offset(row, piece));
      if (c + 8 <= a.n) {
        *reinterpret_cast<uint4*>(p) = u;
      } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < a.n) reinterpret_cast<uint16_t*>(p)[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
      }
    }
  } else {
    for (int row = 0; row < 32 && row0 + row < a.rows; ++row)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = h * 32 + lane, c = c0 + e;
        if (e < cols && c < a.n)
          y[(row0 + row) * a.y_stride + c] =
              reinterpret_cast<const __nv_bfloat16*>(stage + sw128_offset(row, e >> 3))[e & 7];
      }
  }
}

template <int ACT, bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_tiles_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                        const LinearArgs a, const TilesPlan t) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);  // the same place in both CTAs
  __shared__ uint64_t full_bar[kPairStages], empty_bar[kPairStages], tfull_bar[2], tempty_bar[2];
  __shared__ uint32_t tmem_base_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1;
  const int n_tiles = t.wt * t.xt;
  const int mine = pair < n_tiles ? (n_tiles - 1 - pair) / t.pairs + 1 : 0;  // this pair's tiles

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&full_bar[s], 1);   // rank 0's: its expectation, and the bytes of both CTAs
      mbar_init(&empty_bar[s], 1);  // both: the MMAs that read the stage
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], 8);  // rank 0's: the four epilogue warps of both CTAs
    }
    fence_barrier_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive_release();  // both CTAs' barriers are there
  cluster_wait_acquire();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  if (warp == 0) {
    if (lane == 0) {
      griddep_wait();
      griddep_launch_dependents();
      const int half_w = t.bn / 2;
      const uint32_t bytes = 2u * (kHalfBytes + half_w * kBK * 2);
      bool ok = true;
      int q = 0;
      for (int i = 0; i < mine && ok; ++i) {
        const int tile = pair + i * t.pairs;
        const int w0 = tile % t.wt * t.bn + rank * half_w, x0 = tile / t.wt * kPairRows + rank * 128;
        for (int kb = 0; kb < t.boxes; ++kb, ++q) {
          const int s = q % kPairStages;
          if (q >= kPairStages && !mbar_wait(&empty_bar[s], (q / kPairStages - 1) & 1)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[s], bytes);
          const uint32_t bar = mapa_shared(smem_u32(&full_bar[s]), 0);
          uint8_t* st = smem + s * kPairStage;
          tma_load_2d_pair(st, &tm_x, bar, kb * kBK, x0);  // rows past x's, and W's, read 0
          tma_load_2d_pair(st + kHalfBytes, &tm_w, bar, kb * kBK, w0);
        }
      }
      if (!ok) report_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = umma_idesc_bf16(256, t.bn);
      const int total = mine * t.boxes;
      bool ok = true;
      int q = 0;
      for (int i = 0; i < mine && ok; ++i) {
        const int buf = i & 1;
        if (i >= 2 && !mbar_wait_pair(&tempty_bar[buf], ((i >> 1) - 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + buf * 256;
        for (int kb = 0; kb < t.boxes; ++kb, ++q) {
          const int s = q % kPairStages;
          if (!mbar_wait(&full_bar[s], (q / kPairStages) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + s * kPairStage), sb = sa + kHalfBytes;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            umma_bf16_pair(d, umma_desc_sw128(sa + kk * 32), umma_desc_sw128(sb + kk * 32), idesc,
                           (kb > 0 || kk > 0) ? 1u : 0u);
          if (q + kPairStages < total) umma_commit_pair(&empty_bar[s]);  // the last ones no load waits for
        }
        umma_commit_pair(&tfull_bar[buf]);
      }
      if (!ok) report_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    const int quad = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    uint8_t* stage0 = smem + kPairStages * kPairStage + quad * 2 * kStageTile;
    const bool bias_vec = a.bias != nullptr && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    const bool has_r = a.residual != nullptr;
    const int out_bn = GATED ? t.bn / 2 : t.bn;
    bool ok = true;
    griddep_wait();
    for (int i = 0; i < mine; ++i) {
      const int buf = i & 1, tile = pair + i * t.pairs;
      const int w0 = tile % t.wt * t.bn, n0 = GATED ? w0 / 2 : w0;
      const int64_t row0 = static_cast<int64_t>(tile / t.wt) * kPairRows + rank * 128 + quad * 32;
      const int cols = min(out_bn, a.n - n0);  // of y
      if (has_r) residual_to_stage(a, t.r_vec, stage0, row0, n0, cols, lane);
      if (ok && !mbar_wait(&tfull_bar[buf], (i >> 1) & 1)) {
        report_error(a.err, kErrTimeout);
        ok = false;
      }
      tc_fence_after();
      for (int c0 = 0, sb = 0; c0 < cols; c0 += kStageCols, sb ^= 1) {
        uint8_t* st = stage0 + sb * kStageTile;
        if (has_r) {
          if (c0 + kStageCols < cols) {
            residual_to_stage(a, t.r_vec, stage0 + (sb ^ 1) * kStageTile, row0, n0 + c0 + kStageCols,
                              cols - c0 - kStageCols, lane);
            cp_async_wait<1>();
          } else {
            cp_async_wait<0>();
          }
          __syncwarp();
        }
        // 32 columns of the accumulator at a time: 32 or (gated) 16 of y
        constexpr int kOut = GATED ? 16 : 32;
        for (int o0 = 0; o0 < kStageCols && c0 + o0 < cols; o0 += kOut) {
          const int ac = GATED ? 2 * (c0 + o0) : c0 + o0;  // column of the accumulator
          float v[32];
          tmem_ld_32x32b_x32(lanes + buf * 256 + ac, v);
          if (a.bias != nullptr) {
            const __nv_bfloat16* bp = static_cast<const __nv_bfloat16*>(a.bias) + w0 + ac;
            if (bias_vec && w0 + ac + 32 <= a.wide) {
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(bp) + g);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  v[8 * g + 2 * e] += __uint_as_float(w[e] << 16);
                  v[8 * g + 2 * e + 1] += __uint_as_float(w[e] & 0xFFFF0000u);
                }
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (w0 + ac + e < a.wide) v[e] += __bfloat162float(bp[e]);
            }
          }
          float o[kOut];
#pragma unroll
          for (int e = 0; e < kOut; ++e) o[e] = GATED ? activate<ACT>(v[2 * e]) * v[2 * e + 1] : activate<ACT>(v[e]);
#pragma unroll
          for (int g = 0; g < kOut / 8; ++g) {
            uint4* p = reinterpret_cast<uint4*>(st + sw128_offset(lane, o0 / 8 + g));
            if (has_r) {
              const uint4 u = *p;
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[8 * g + 2 * e] += __uint_as_float(w[e] << 16);
                o[8 * g + 2 * e + 1] += __uint_as_float(w[e] & 0xFFFF0000u);
              }
            }
            *p = make_uint4(pack_bf16x2(o[8 * g], o[8 * g + 1]), pack_bf16x2(o[8 * g + 2], o[8 * g + 3]),
                            pack_bf16x2(o[8 * g + 4], o[8 * g + 5]), pack_bf16x2(o[8 * g + 6], o[8 * g + 7]));
          }
        }
        if (c0 + kStageCols >= cols) {  // the accumulator is read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(mapa_shared(smem_u32(&tempty_bar[buf]), 0));
        }
        __syncwarp();
        stage_to_y(a, t.y_vec, st, row0, n0 + c0, min(kStageCols, cols - c0), lane);
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive_release();  // nothing of the other CTA's is on its way here any more
  cluster_wait_acquire();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ------------------------------------------------------------ host
RowsPlan rows_plan(const LinearArgs& a, int bn, int split, int ring_bytes) {
  RowsPlan t;
  t.bn = bn;
  t.split = split;
  t.boxes = (a.k + kBK - 1) / kBK;
  const int stage = kABytes + bn * kBK * 2;
  const int share = (t.boxes + split - 1) / split;
  t.stages = ring_bytes / stage;
  t.stages = t.stages > kMaxStages ? kMaxStages : t.stages;
  t.stages = t.stages > share ? share : t.stages;
  t.per_rank = (bn / 4 + split - 1) / split;
  t.cols = 32;
  while (t.cols < static_cast<uint32_t>(bn)) t.cols *= 2;
  t.xt = (a.rows + bn - 1) / bn;
  return t;
}

template <int ACT, bool GATED>
cudaError_t launch_rows(const LinearArgs& a, const RowsPlan& t, cudaStream_t stream) {
  CUtensorMap tm_w, tm_x;
  cudaError_t e = encode_rows_sw128(&tm_w, a.w, a.k, a.wide, a.k, kBK, kTW);
  if (e == cudaSuccess)
    e = a.gain != nullptr ? encode_rows_sw128(&tm_x, a.xhat, a.k, a.rows, a.k, kBK, t.bn)
                          : encode_rows_sw128(&tm_x, a.x, a.k, a.rows, a.x_stride, kBK, t.bn);
  if (e != cudaSuccess) return e;
  int smem = t.stages * (kABytes + t.bn * kBK * 2);
  const int join = t.split > 1 ? t.split * t.per_rank * kTW * 16 : 0;
  smem = (smem > join ? smem : join) + 1024;
  e = cudaFuncSetAttribute(linear_rows_kernel<ACT, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.wide + kTW - 1) / kTW) * t.xt * t.split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = t.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_rows_kernel<ACT, GATED>, tm_w, tm_x, a, t);
}

bool rows16(const void* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0; }

template <int ACT, bool GATED>
cudaError_t launch_tiles(const LinearArgs& a, int bn, int num_sms, cudaStream_t stream) {
  TilesPlan t;
  t.bn = bn;
  t.boxes = (a.k + kBK - 1) / kBK;
  t.wt = (a.wide + bn - 1) / bn;
  t.xt = (a.rows + kPairRows - 1) / kPairRows;
  t.pairs = num_sms / 2;
  if (t.pairs > t.wt * t.xt) t.pairs = t.wt * t.xt;
  t.y_vec = rows16(a.y, a.y_stride);
  t.r_vec = a.residual != nullptr && rows16(a.residual, a.r_stride);
  CUtensorMap tm_w, tm_x;
  cudaError_t e = encode_rows_sw128(&tm_w, a.w, a.k, a.wide, a.k, kBK, bn / 2);
  if (e == cudaSuccess)
    e = a.gain != nullptr ? encode_rows_sw128(&tm_x, a.xhat, a.k, a.rows, a.k, kBK, 128)
                          : encode_rows_sw128(&tm_x, a.x, a.k, a.rows, a.x_stride, kBK, 128);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(linear_tiles_kernel<ACT, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * t.pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_tiles_kernel<ACT, GATED>, tm_w, tm_x, a, t);
}

template <int ACT, bool GATED>
cudaError_t launch_product(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  const int boxes = (a.k + kBK - 1) / kBK;
  if (a.rows > 256) return launch_tiles<ACT, GATED>(a, 256, num_sms, stream);
  const int bn = (a.rows + 15) / 16 * 16;
  int split = num_sms / ((a.wide + kTW - 1) / kTW);
  split = split < 1 ? 1 : split > kMaxSplit ? kMaxSplit : split;
  split = split > boxes ? boxes : split;
  return launch_rows<ACT, GATED>(a, rows_plan(a, bn, split, 200 * 1024), stream);
}

template <int ACT>
cudaError_t launch_act(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  return a.gated ? launch_product<ACT, true>(a, num_sms, stream) : launch_product<ACT, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream) {
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
