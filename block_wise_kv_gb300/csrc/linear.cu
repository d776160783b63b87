// linear.cu — products with a weight: y = act(x^ W^T + b) + r, also of gate and up units
// side by side, on tcgen05 (sm_103a).
//
//  * linear_norm_kernel  x^ = RMSNorm(x), correctly rounded to bf16, 32 to 256 threads a row
//    (only where the call has a gain, and rows are not so few that the product norms them).
//  * linear_few_kernel   one or two rows (linear_few.cu).
//  * linear_rows_kernel  few rows: 128 rows of W are the tensor core's M, up to 128 rows of
//    x its N.  K is cut over the CTAs of a cluster, so that all SMs read W; each CTA's sums go
//    to the one that finishes them, 16 bytes a store, counted by a barrier there, and are
//    added in the order of K.  Warps 0 and 6 stream boxes of 64 columns of W and x through a
//    ring, warp 1 issues the MMAs into TMEM, warps 2-5 make y (a thread: one row of W; a warp's
//    32 neighbouring columns of y are one 64-byte run).
//  * linear_tiles_kernel many rows: a pair of CTAs (cta_group::2) takes 256 rows of x by up
//    to 256 rows of W, each CTA half of either operand, and walks such tiles.  Two
//    accumulators in TMEM: warps 2-9 of each CTA make y of one tile (a thread: one row of x)
//    while the tensor cores work on the next, through staging tiles that make whole runs of
//    the rows of y and of the residual.
//
// The tensor core's sums go over all of K (or of a CTA's part): one in 140 values of y of K = 12288
// is the neighbour of the nearest bf16, one in 240 of K = 4096 gated, and the error against 64 bits is
// that of an fp32 product (relative 1.66e-3, all of it y's rounding).
//
// Bound and measured (us, calls one behind the other, W from memory).  64 rows, 4096 x 4096:
// 11.2 (floor 5.2; 9.0 with W in L2): W comes at 6 TB/s in 5.6 of it, the rest is the first box's way
// (1.3), the parts' (2), and from a kernel's end to the next one's start (1.2).  512 rows, K 4096, 2 x
// 12288 gated and normed: 66.5 (53.7), of which the norm is 3: tensor pipe 75% busy, held up by
// what L2 delivers (14.5 TB/s for all SMs; 256 x 224 tiles need 60 KB for 0.24 us of MMAs).
// 20480 rows, K 12288, 4096: 1056 to 1100 in a burst (1073), 1256 at the clock that the power
// limit leaves (the measured sustained rate: 1207).  Library products of the first two's sizes:
// 8.2 and 65.
//
// The waits sleep without reading the timer as mbar_wait does: reading it, or trying more
// often, slows the CTA down (prompts 1179, 1190, gated 87, 87).  Lines of W asked for ahead,
// as far as L2, by the copy engine or by idle warps, before or behind the wait for the kernel
// in front, made every case slower.
#include <math.h>

#include "linear_math.cuh"
#include "sm103.cuh"
#include "tmap.cuh"

namespace dllm {
namespace {

// ------------------------------------------------------------ RMSNorm
constexpr int kNormThreads = 256;

// A row to TEAM threads, each with up to four pieces of 8 elements in registers; what is behind those is read twice.
template <int TEAM>
__global__ void __launch_bounds__(kNormThreads) linear_norm_kernel(const LinearArgs a) {
  constexpr int kTeams = kNormThreads / TEAM, kHeld = 4;
  __shared__ float2 part[kNormThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nvec = a.k / 8;
  griddep_launch_dependents();  // the product behind reads nothing before its own wait
  griddep_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + threadIdx.x / TEAM;
  const bool there = row < a.rows;
  const int l = there ? threadIdx.x % TEAM : nvec;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + (there ? row : 0) * a.x_stride);
  uint4* out = static_cast<uint4*>(a.xhat) + row * nvec;
  const uint4* g = static_cast<const uint4*>(a.gain);
  uint4 u[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) u[i] = l + i * TEAM < nvec ? __ldg(x + l + i * TEAM) : make_uint4(0u, 0u, 0u, 0u);
  float2 hi2 = {0.f, 0.f}, lo2 = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (l + i * TEAM < nvec) sumsq2_add(u[i], hi2, lo2);
  for (int v = l + kHeld * TEAM; v < nvec; v += TEAM) sumsq2_add(__ldg(x + v), hi2, lo2);
  float hi, lo;
  sums_of(hi2, lo2, hi, lo);
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    const float oh = __shfl_xor_sync(0xffffffffu, hi, o), ol = __shfl_xor_sync(0xffffffffu, lo, o);
    pair_add(hi, lo, oh, ol);
  }
  hi = __shfl_sync(0xffffffffu, hi, 0);  // lane 0's sum is the warp's
  lo = __shfl_sync(0xffffffffu, lo, 0);
  if (TEAM > 32) {
    if (lane == 0) part[warp] = make_float2(hi, lo);
    __syncthreads();
    const int w0 = threadIdx.x / TEAM * (TEAM / 32);
    hi = part[w0].x;
    lo = part[w0].y;
    for (int w = 1; w < TEAM / 32; ++w) pair_add(hi, lo, part[w0 + w].x, part[w0 + w].y);
  }
  two_sum(hi, lo, hi, lo);
  float s_hi, s_lo;
  rsqrt_pair(hi, lo, a.k, a.rms_eps, s_hi, s_lo);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int v = l + i * TEAM;
    if (v < nvec) out[v] = normed8(u[i], __ldg(g + v), s_hi, s_lo);
  }
  for (int v = l + kHeld * TEAM; v < nvec; v += TEAM) out[v] = normed8(__ldg(x + v), __ldg(g + v), s_hi, s_lo);
}

// ------------------------------------------------------------ few rows
constexpr int kThreads = 224;       // warps: W, MMAs, four that make y, x
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
  int norm;       // the normed x of this CTA's part of K is made here: where in shared memory, or 0
  int per_rank;   // groups of 4 rows of x that each CTA of a cluster finishes
  int join;       // where in shared memory the parts of a tile meet: behind the ring, or 0, in the ring when that is done with
  int smem;       // dynamic shared memory
  uint32_t cols;  // TMEM columns
  int xt;         // tiles of x
};

// A bounded wait without the timer that mbar_wait reads.  A try at a phase that is not over takes 3.8 us, whatever time up to
// 100 us it is given: two seconds and more in all.  (The timer behind every thousand tries, inlined or in a function of its
// own: 64 rows 10.8 us for 10.7, gated 77.7 for 76.8.)
constexpr int kTries = 600000;
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int tries = kTries) {
#pragma unroll 1
  for (int i = 0; i < tries; ++i)
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
  return false;
}
// As that, for a warp that begins to wait while the kernel in front may still run: only what runs out behind that is this
// kernel's own.  (Waiting for that kernel first: 777 rows of 1000 x 1003 11.26 us for 11.13.)
__device__ __forceinline__ bool wait_box(uint64_t* bar, uint32_t parity) {
  if (wait_phase(bar, parity)) return true;
  griddep_wait();
  return wait_phase(bar, parity);
}
// For what comes once all boxes of a tile are there: one takes 0.3 us.
__device__ __forceinline__ int tries_of(int boxes) { return kTries + boxes; }

// A place in a ring and the parity of its present use, stepped without divisions: a division by the number of stages costs
// the one thread that issues the loads about as much as the load (an SM's loads then came at 51 GB/s, not at 100).
struct Ring {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      parity ^= 1;
    }
  }
};

// 16 bytes to a place in the shared memory of a CTA of the cluster, counted by the barrier there.
__device__ __forceinline__ void st_async_v4(uint32_t addr, float x, float y, float z, float w, uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr), "f"(x),
      "f"(y), "f"(z), "f"(w), "r"(bar)
      : "memory");
}

// Sixteen rows of x (row, row + 1, ...) under this thread's row of W: what is added to y, asked for ahead, and y from
// the sums v.  Gated, the even lane has the gate of the sixteen and the odd one the up: each makes y of eight.
template <bool GATED>
struct Finish {
  static constexpr int kOut = GATED ? 8 : 16;
  __nv_bfloat16 r[kOut];

  static __device__ __forceinline__ int64_t row_of(int row, int i, int lane) { return row + (GATED ? (lane & 1) * 8 : 0) + i; }

  __device__ __forceinline__ void ask(const LinearArgs& a, int wr, int row, int lane) {
    const int n = GATED ? wr >> 1 : wr;
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
      const int64_t j = row_of(row, i, lane);
      r[i] = __float2bfloat16_rn(0.f);
      if (a.residual != nullptr && wr < a.wide && j < a.rows)
        r[i] = static_cast<const __nv_bfloat16*>(a.residual)[j * a.r_stride + n];
    }
  }

  template <int ACT>
  __device__ __forceinline__ void make(const LinearArgs& a, const float (&v)[16], float b, int wr, int row, int lane,
                                       int end = 0x7fffffff) {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y);
    const bool up = lane & 1;
    const int n = GATED ? wr >> 1 : wr;
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
      float o;
      if (GATED) {
        const float mine = (up ? v[8 + i] : v[i]) + b, give = (up ? v[i] : v[8 + i]) + b;
        const float other = __shfl_xor_sync(0xffffffffu, give, 1);
        o = activate<ACT>(up ? other : mine) * (up ? mine : other);
      } else {
        o = activate<ACT>(v[i] + b);
      }
      const int64_t j = row_of(row, i, lane);
      if (wr < a.wide && j < a.rows && j < end) y[j * a.y_stride + n] = __float2bfloat16_rn(o + __bfloat162float(r[i]));
    }
  }
};

// Threads that norm a row inside the product: four pieces of 8 elements each (fewer: a piece's eight exact squares are a
// chain of eight sums).
constexpr int kNormPieces = 4;
__host__ __device__ inline int norm_lanes(int k) {
  int t = 8;
  while (t * kNormPieces * 8 < k) t *= 2;
  return t;
}
constexpr int kNormThreadsInside = 128;

// Four warps (tid: 0 to 127): columns [64 kb0, 64 (kb0 + nb)) of RMSNorm(x) of the rows from x0 on, as the boxes that the
// MMAs take (rows of 128 bytes, swizzled).  `boxes` is zero where no row or column is.
__device__ __forceinline__ void norm_rows(const LinearArgs& a, uint8_t* boxes, int x0, int bn, int kb0, int nb, int tid) {
  const int nvec = a.k / 8, lanes = norm_lanes(a.k), sub = tid / lanes, l = tid % lanes;
  const uint4* g = static_cast<const uint4*>(a.gain);
  const int rows = min(bn, a.rows - x0);
  for (int r0 = 0; r0 < rows; r0 += kNormThreadsInside / lanes) {
    const int row = r0 + sub;
    const bool there = row < rows;
    const uint4* x =
        reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + (x0 + (there ? row : 0)) * a.x_stride);
    uint4 u[kNormPieces], w[kNormPieces];
#pragma unroll
    for (int i = 0; i < kNormPieces; ++i) {
      const int v = l + i * lanes;
      u[i] = w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (v < nvec) u[i] = __ldg(x + v);
      if (v >= kb0 * 8 && v < (kb0 + nb) * 8 && v < nvec) w[i] = __ldg(g + v);
    }
    float2 hi2 = {0.f, 0.f}, lo2 = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kNormPieces; ++i) sumsq2_add(u[i], hi2, lo2);
    float hi, lo;
    sums_of(hi2, lo2, hi, lo);
    for (int o = 1; o < lanes; o <<= 1) {
      const float oh = __shfl_xor_sync(0xffffffffu, hi, o), ol = __shfl_xor_sync(0xffffffffu, lo, o);
      // (the same order in both lanes: the pair sum is not commutative in its last bits)
      float h = (tid & o) ? oh : hi, s = (tid & o) ? ol : lo;
      pair_add(h, s, (tid & o) ? hi : oh, (tid & o) ? lo : ol);
      hi = h;
      lo = s;
    }
    two_sum(hi, lo, hi, lo);
    float s_hi, s_lo;
    rsqrt_pair(hi, lo, a.k, a.rms_eps, s_hi, s_lo);
#pragma unroll
    for (int i = 0; i < kNormPieces; ++i) {
      const int v = l + i * lanes, c = v - kb0 * 8;
      if (there && c >= 0 && c < nb * 8 && v < nvec)
        *reinterpret_cast<uint4*>(boxes + (c >> 3) * bn * 128 + sw128_offset(row, c & 7)) = normed8(u[i], w[i], s_hi, s_lo);
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
  __shared__ uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], done_bar, join_bar, norm_bar;
  __shared__ uint32_t tmem_base_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x_box = t.bn * kBK * 2, stage_bytes = kABytes + (t.norm ? 0 : x_box);
  const int rank = static_cast<int>(blockIdx.x) % t.split, tile = static_cast<int>(blockIdx.x) / t.split;
  const int w0 = tile / t.xt * kTW, x0 = tile % t.xt * t.bn;  // tiles that share rows of W side by side
  const int kb0 = static_cast<int>(static_cast<int64_t>(t.boxes) * rank / t.split);
  const int nb = static_cast<int>(static_cast<int64_t>(t.boxes) * (rank + 1) / t.split) - kb0;
  const int groups = t.split > 1 ? min(t.per_rank, t.bn / 4 - rank * t.per_rank) : 0;  // that this CTA finishes, of 4 rows of x

  if (threadIdx.x == 0) {
    for (int s = 0; s < t.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&done_bar, 1);
    mbar_init(&join_bar, 1);
    mbar_init(&norm_bar, 4);
    fence_barrier_init();
    if (groups > 0) mbar_arrive_expect_tx(&join_bar, t.split * groups * kTW * 16);
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) tmem_alloc(&tmem_base_sh, t.cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (t.split > 1 && t.join > 0) cluster_arrive_release();  // this CTA's barrier and buffer are there
  const uint32_t tmem = tmem_base_sh;
  const int quad = warp & 3;
  const int wr = w0 + quad * 32 + lane;  // warps 2-5: this thread's row of W
  float b = 0.f;
  Finish<GATED> fin;
  const int first = t.split > 1 ? rank * t.per_rank * 4 : 0;  // the first row of x that this CTA finishes

  if (warp == 0 || warp == 6) {
    // Warp 0 loads W, warp 6 x: a thread's next load goes out some 100 ns behind the one before.
    if (lane == 0 && (warp == 0 || t.norm == 0)) {
      const bool is_w = warp == 0;
      const CUtensorMap* map = is_w ? &tm_w : &tm_x;
      const int y0 = is_w ? w0 : x0;
      uint8_t* dst = smem + (is_w ? 0 : kABytes);
      bool ok = true;
      griddep_wait();
      griddep_launch_dependents();
      Ring r;
      int i = 0;
      for (; i < nb; ++i, r.next(t.stages)) {
        if (i >= t.stages && !wait_phase(&empty_bar[r.s], r.parity ^ 1)) {
          ok = false;
          break;
        }
        if (is_w) mbar_arrive_expect_tx(&full_bar[r.s], stage_bytes);
        tma_load_2d(dst + r.s * stage_bytes, map, &full_bar[r.s], (kb0 + i) * kBK, y0);  // rows past the last read 0
      }
      // every load has landed before the ring ends: each place's last one
      for (int j = 0; j < t.stages && j < i; ++j, r.next(t.stages))
        ok = wait_phase(&full_bar[i < t.stages ? j : r.s], i < t.stages ? 0 : r.parity ^ 1) && ok;
      if (!ok) report_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = umma_idesc_bf16(kTW, t.bn);
      bool ok = t.norm == 0 || wait_box(&norm_bar, 0);
      Ring r;
      for (int i = 0; i < nb && ok; ++i, r.next(t.stages)) {
        ok = wait_box(&full_bar[r.s], r.parity);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem) + r.s * stage_bytes;
        const uint32_t sb = t.norm ? smem_u32(smem) + t.norm + i * x_box : sa + kABytes;
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          umma_bf16(tmem, umma_desc_sw128(sa + kk * 32), umma_desc_sw128(sb + kk * 32), idesc,
                    (i > 0 || kk > 0) ? 1u : 0u);
        if (i + t.stages < nb) umma_commit(&empty_bar[r.s]);  // the last ones no load waits for
      }
      umma_commit(&done_bar);
      if (!ok) report_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    if (t.norm)
      for (int i = threadIdx.x - 64; i < nb * x_box / 16; i += 128)
        reinterpret_cast<uint4*>(smem + t.norm)[i] = make_uint4(0u, 0u, 0u, 0u);
    griddep_wait();  // bias, residual, and y behind whoever reads it
    b = wr < a.wide && a.bias != nullptr ? bf16_at(a.bias, wr) : 0.f;
    if (t.norm) {
      named_barrier(1, 128);
      norm_rows(a, smem + t.norm, x0, t.bn, kb0, nb, threadIdx.x - 64);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read it
      __syncwarp();
      if (lane == 0) mbar_arrive(&norm_bar);
    }
    fin.ask(a, wr, x0 + first, lane);
    if (!wait_phase(&done_bar, 0, tries_of(nb))) report_error(a.err, kErrTimeout);
    tc_fence_after();
  }
  const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  if (t.split == 1) {
    if (warp >= 2 && warp < 6) {
      for (int c0 = 0; c0 < t.bn && x0 + c0 < a.rows; c0 += 16) {
        float v[16];
        tmem_ld_32x32b_x16(src + c0, v);
        Finish<GATED> next;
        if (c0 + 16 < t.bn) next.ask(a, wr, x0 + c0 + 16, lane);
        fin.template make<ACT>(a, v, b, wr, x0 + c0, lane);
        fin = next;
      }
    }
  } else {
    // Each CTA's sums of group g (four rows of x) go to the CTA that finishes it: [CTA they come from][group][row of W],
    // 16 bytes each, counted there.
    if (t.join == 0) {  // into the rings, once they are done with on all sides
      __syncthreads();
      cluster_arrive_release();
    }
    cluster_wait_acquire();
    if (warp >= 2 && warp < 6) {
      const uint32_t mine = smem_u32(smem) + t.join + (quad * 32 + lane) * 16;
      int g = 0, to = 0;  // the group within those of CTA `to`
      for (int c0 = 0; c0 < t.bn; c0 += 16) {
        float v[16];
        tmem_ld_32x32b_x16(src + c0, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int there = min(t.per_rank, t.bn / 4 - to * t.per_rank);
          st_async_v4(mapa_shared(mine + (rank * there + g) * (kTW * 16), to), v[4 * i], v[4 * i + 1], v[4 * i + 2],
                      v[4 * i + 3], mapa_shared(smem_u32(&join_bar), to));
          if (++g == there) {
            g = 0;
            ++to;
          }
        }
      }
      if (groups > 0) {
        // (a CTA that gave a wait up sends all the same: not before all have is this one's shared memory let go)
        if (!wait_phase(&join_bar, 0, 2 * tries_of(nb))) report_error(a.err, kErrTimeout);
        const float4* part = reinterpret_cast<const float4*>(smem + t.join) + quad * 32 + lane;
        const int end = first + groups * 4;
        for (int c0 = first, g0 = 0; c0 < end && x0 + c0 < a.rows; c0 += 16, g0 += 4) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.f;
          for (int r = 0; r < t.split; ++r) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (g0 + i >= groups) break;
              const float4 p = part[(r * groups + g0 + i) * kTW];
              v[4 * i] += p.x;
              v[4 * i + 1] += p.y;
              v[4 * i + 2] += p.z;
              v[4 * i + 3] += p.w;
            }
          }
          Finish<GATED> next;
          if (c0 + 16 < end) next.ask(a, wr, x0 + c0 + 16, lane);
          fin.template make<ACT>(a, v, b, wr, x0 + c0, lane, x0 + end);
          fin = next;
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

// ------------------------------------------------------------ many rows
constexpr int kPairRows = 256;           // rows of x to a pair's tile
constexpr int kPairStages = 6;
constexpr int kHalfBytes = 128 * kBK * 2;  // a CTA's half of an operand's box, at most
constexpr int kPairStage = 2 * kHalfBytes;
constexpr int kStageCols = 64;           // columns of y in a staging tile: 128-byte rows
constexpr int kStageTile = 32 * kStageCols * 2;
constexpr int kPairWarps = 8;           // that make y: two to a quadrant of TMEM's lanes, every other kStageCols columns each
constexpr int kPairThreads = 32 * (kPairWarps + 3);
constexpr int kPairSmem = kPairStages * kPairStage + kPairWarps * kStageTile + 1024;

struct TilesPlan {
  int bn;      // rows of W to a tile: a multiple of 32, at most 256
  int boxes;   // of K
  int wt, xt;  // tiles of W, of x
  int pairs;   // CTA pairs
  int band;    // tiles of x that are walked side by side
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
  const bool ok = wait_phase(bar, parity);
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

// Rows that do not lie on 16-byte boundaries go two elements a lane: those of a word, or, where the row begins in the middle
// of one, of the words behind that and (the last lane) the two at its ends.  With an odd stride every second row does.
struct Pair {
  int a, b;
  bool word, one_a, one_b;  // both as a word, or one by one
  __device__ __forceinline__ Pair(int odd, int lane, int n) {
    const bool ends = odd && lane == 31;
    a = ends ? 0 : 2 * lane + odd;
    b = ends ? kStageCols - 1 : a + 1;
    word = !ends && b < n;
    one_a = !word && a < n;
    one_b = !word && b < n;
  }
};
__device__ __forceinline__ int odd_address(const void* p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1) & 1; }
__device__ __forceinline__ uint16_t* at_stage(uint8_t* stage, int row, int e) {
  return reinterpret_cast<uint16_t*>(stage + sw128_offset(row, e >> 3)) + (e & 7);
}

// The residual of kStageCols columns of 32 rows, as a warp asks for it and then has it in its staging tile (rows of 128
// bytes, 16-byte pieces swizzled by the row).  Rows on 16-byte boundaries come in pieces.  Others come in words: where a row
// begins in the middle of one, element e lies at place e + 1, the last at place 0, and the elements that share a word with
// another row's or chunk's come through a register of the row's lane.
struct Residual {
  uint32_t first, last;
  int n, rows;

  static __device__ __forceinline__ int odd(const void* p) { return odd_address(p); }

  // p: the chunk's first element of the first row; cols: columns that exist
  __device__ __forceinline__ void ask(const LinearArgs& a, bool vec, uint8_t* stage, const uint16_t* p, int64_t row0, int cols,
                                      int lane) {
    n = min(kStageCols, cols);
    rows = static_cast<int>(a.rows - row0 < 32 ? a.rows - row0 : 32);
    if (vec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = i * 4 + lane / 8, e = (lane & 7) * 8;
        if (row >= rows || e >= n) continue;
        const uint16_t* from = p + row * a.r_stride + e;
        if (e + 8 <= n) {
          cp_async16(smem_u32(stage) + sw128_offset(row, lane & 7), from);
        } else {
          for (int k = 0; e + k < n; ++k) at_stage(stage, row, e)[k] = from[k];
        }
      }
    } else {
      const int o_even = odd(p), o_odd = odd(p + a.r_stride);
      const uint16_t* from = p;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i, from += a.r_stride) {
          const int o = i & 1 ? o_odd : o_even, e = 2 * lane + o, at = e + o;
          const uint32_t to = smem_u32(stage) + (r0 + i) * 128 + (((at >> 3) << 4) ^ (i << 4)) + (at & 7) * 2;
          if (r0 + i < rows && e + 1 < n)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from + e) : "memory");
        }
      }
      from = p + lane * a.r_stride;
      const int o = odd(from);
      first = last = 0;
      if (lane < rows && o) first = from[0];
      if (lane < rows && ((n ^ o) & 1)) last = from[n - 1];
    }
    cp_async_commit();
  }
  __device__ __forceinline__ void settle(const LinearArgs& a, bool vec, uint8_t* stage, const uint16_t* p, int lane) {
    cp_async_wait<0>();
    if (!vec && lane < rows) {
      const int o = odd(p + lane * a.r_stride);
      if (o) *at_stage(stage, lane, 1) = static_cast<uint16_t>(first);
      if ((n ^ o) & 1) *at_stage(stage, lane, (n - 1 + o) & (kStageCols - 1)) = static_cast<uint16_t>(last);
    }
    __syncwarp();
  }
};

// kStageCols columns of 32 rows of y out of a warp's staging tile.
__device__ __forceinline__ void stage_to_y(const LinearArgs& a, bool vec, uint8_t* stage, int64_t row0, int c0, int cols,
                                           int lane) {
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
    const int rows = static_cast<int>(a.rows - row0 < 32 ? a.rows - row0 : 32), n = min(cols, a.n - c0);
    uint16_t* p = reinterpret_cast<uint16_t*>(y) + row0 * a.y_stride + c0;
    const Pair even(odd_address(p), lane, n), odd(odd_address(p + a.y_stride), lane, n);  // of the rows 0, 2, ... and 1, 3, ...
#pragma unroll 1
    for (int from = 0; from < rows; from += 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i, p += a.y_stride) {
        const Pair& e = i & 1 ? odd : even;
        // (the address of at_stage, the row's swizzle being i's)
        const uint8_t* base = stage + from * 128 + i * 128;
        const uint16_t va = *reinterpret_cast<const uint16_t*>(base + (((e.a >> 3) << 4) ^ (i << 4)) + (e.a & 7) * 2);
        const uint16_t vb = *reinterpret_cast<const uint16_t*>(base + (((e.b >> 3) << 4) ^ (i << 4)) + (e.b & 7) * 2);
        if (from + i >= rows) continue;
        if (e.word) *reinterpret_cast<uint32_t*>(p + e.a) = va | static_cast<uint32_t>(vb) << 16;
        if (e.one_a) p[e.a] = va;
        if (e.one_b) p[e.b] = vb;
      }
    }
  }
}

// Tiles in bands of t.band tiles of x (the last may be narrower); within a band tile of W by tile of W, so that those who
// work side by side share tiles of both.
__device__ __forceinline__ void tile_at(const TilesPlan& t, int tile, int& wt, int& xt) {
  const int per = t.band * t.wt, b = tile / per, rest = tile - b * per;
  const int width = min(t.band, t.xt - b * t.band);
  wt = rest / width;
  xt = b * t.band + rest % width;
}

template <int ACT, bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
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
      mbar_init(&tempty_bar[i], 2 * kPairWarps);  // rank 0's: the warps of both CTAs that read it
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

  if (warp == 0 || warp == kPairWarps + 2) {
    if (lane == 0) {  // (as above) warp 0 loads W, the last one x
      const bool is_w = warp == 0;
      const int half_w = t.bn / 2;
      const uint32_t bytes = 2u * (kHalfBytes + half_w * kBK * 2);
      const uint32_t full0 = mapa_shared(smem_u32(&full_bar[0]), 0);
      const CUtensorMap* map = is_w ? &tm_w : &tm_x;
      uint8_t* dst = smem + (is_w ? kHalfBytes : 0);
      griddep_wait();
      griddep_launch_dependents();
      bool ok = true;
      Ring r;
      int q = 0;
      for (int i = 0; i < mine && ok; ++i) {
        int wt, xt;
        tile_at(t, pair + i * t.pairs, wt, xt);
        const int y0 = is_w ? wt * t.bn + rank * half_w : xt * kPairRows + rank * 128;
        for (int kb = 0; kb < t.boxes; ++kb, ++q, r.next(kPairStages)) {
          if (q >= kPairStages && !wait_phase(&empty_bar[r.s], r.parity ^ 1)) {
            ok = false;
            break;
          }
          if (is_w && rank == 0) mbar_arrive_expect_tx(&full_bar[r.s], bytes);
          tma_load_2d_pair(dst + r.s * kPairStage, map, full0 + r.s * 8, kb * kBK, y0);  // rows past the last read 0
        }
      }
      if (!ok) report_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = umma_idesc_bf16(256, t.bn);
      griddep_wait();
      const int total = mine * t.boxes;
      bool ok = true;
      Ring r;
      int q = 0;
      for (int i = 0; i < mine && ok; ++i) {
        const int buf = i & 1;
        if (i >= 2 && !mbar_wait_pair(&tempty_bar[buf], ((i >> 1) - 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + buf * 256;
        for (int kb = 0; kb < t.boxes; ++kb, ++q, r.next(kPairStages)) {
          if (!wait_phase(&full_bar[r.s], r.parity)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem) + r.s * kPairStage, sb = sa + kHalfBytes;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            umma_bf16_pair(d, umma_desc_sw128(sa + kk * 32), umma_desc_sw128(sb + kk * 32), idesc,
                           (kb > 0 || kk > 0) ? 1u : 0u);
          if (q + kPairStages < total) umma_commit_pair(&empty_bar[r.s]);  // the last ones no load waits for
        }
        umma_commit_pair(&tfull_bar[buf]);
      }
      if (!ok) report_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    uint8_t* st = smem + kPairStages * kPairStage + (warp - 2) * kStageTile;
    const bool bias_vec = a.bias != nullptr && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    const bool has_r = a.residual != nullptr;
    const int out_bn = GATED ? t.bn / 2 : t.bn;
    Residual res;
    bool ok = true;
    griddep_wait();
    for (int i = 0; i < mine; ++i) {
      const int buf = i & 1;
      int wt, xt;
      tile_at(t, pair + i * t.pairs, wt, xt);
      const int w0 = wt * t.bn, n0 = GATED ? w0 / 2 : w0;
      const int64_t row0 = static_cast<int64_t>(xt) * kPairRows + rank * 128 + quad * 32;
      const int cols = min(out_bn, a.n - n0);  // of y
      const uint16_t* r0 = has_r ? static_cast<const uint16_t*>(a.residual) + row0 * a.r_stride + n0 : nullptr;
      const int first = half * kStageCols;
      const uint32_t empty = mapa_shared(smem_u32(&tempty_bar[buf]), 0);
      if (has_r && first < cols) res.ask(a, t.r_vec, st, r0 + first, row0, cols - first, lane);
      if (ok && !wait_phase(&tfull_bar[buf], (i >> 1) & 1, tries_of(t.boxes))) {
        report_error(a.err, kErrTimeout);
        ok = false;
      }
      tc_fence_after();
      for (int c0 = first; c0 < cols; c0 += 2 * kStageCols) {
        uint32_t shift = 0, last = 0;  // of this lane's row of the residual
        if (has_r) {
          res.settle(a, t.r_vec, st, r0 + c0, lane);
          if (!t.r_vec) {
            shift = Residual::odd(r0 + c0 + lane * a.r_stride);
            last = *at_stage(st, lane, 0);
          }
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
              uint32_t w[4] = {u.x, u.y, u.z, u.w};
              if (shift) {
                const int piece = o0 / 8 + g;
                const uint32_t end = piece == 7 ? last : *at_stage(st, lane, 8 * piece + 8);
                w[0] = w[0] >> 16 | w[1] << 16;
                w[1] = w[1] >> 16 | w[2] << 16;
                w[2] = w[2] >> 16 | w[3] << 16;
                w[3] = w[3] >> 16 | end << 16;
              }
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
        const int c1 = c0 + 2 * kStageCols;
        if (c1 >= cols) tc_fence_before();
        __syncwarp();
        if (c1 >= cols && lane == 0) mbar_arrive_at(empty);  // this warp has read the accumulator
        stage_to_y(a, t.y_vec, st, row0, n0 + c0, min(kStageCols, cols - c0), lane);
        __syncwarp();
        if (has_r && c1 < cols) res.ask(a, t.r_vec, st, r0 + c1, row0, cols - c1, lane);
      }
      if (first >= cols && lane == 0) mbar_arrive_at(empty);
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
bool rows16(const void* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0; }

// Shared memory of a CTA: two fit an SM, so that one's loads go on while the other finishes, and a cluster finds room (one row:
// 12.2 us with 100 KB, 18.5 with 200 KB, where 48 clusters of three do not fit at once; 64 rows 11.9 and 12.0 to 19).
constexpr int kRowsSmem = 108 * 1024;
constexpr int kRowsSmemMost = kRowsSmem + 1024;  // that any plan takes: the ring has two places at least, which fit beside the rest

RowsPlan rows_plan(const LinearArgs& a, int bn, int split, bool norm) {
  RowsPlan t;
  t.bn = bn;
  t.split = split;
  t.boxes = (a.k + kBK - 1) / kBK;
  t.xt = (a.rows + bn - 1) / bn;
  t.per_rank = (bn / 4 + split - 1) / split;
  const int share = (t.boxes + split - 1) / split, x_box = bn * kBK * 2;
  const int join = split > 1 ? split * t.per_rank * kTW * 16 : 0, xhat = norm ? share * x_box : 0;
  const int stage = kABytes + (norm ? 0 : x_box);
  const bool aside = join > 0 && join <= kRowsSmem / 3;  // else the parts meet in the ring
  t.stages = (kRowsSmem - xhat - (aside ? join : 0)) / stage;
  t.stages = t.stages > kMaxStages ? kMaxStages : t.stages < 2 ? 2 : t.stages;
  t.stages = t.stages > share ? share : t.stages;
  t.norm = norm ? t.stages * stage : 0;
  t.join = aside ? t.stages * stage + xhat : 0;
  t.smem = t.stages * stage + xhat;
  t.smem = (aside ? t.smem + join : t.smem > join ? t.smem : join) + 1024;
  t.cols = 32;
  while (t.cols < static_cast<uint32_t>(bn)) t.cols *= 2;
  return t;
}

template <int ACT, bool GATED>
cudaError_t launch_rows(const LinearArgs& a, const RowsPlan& t, cudaStream_t stream) {
  CUtensorMap tm_w, tm_x;
  cudaError_t e = encode_rows_sw128(&tm_w, a.w, a.k, a.wide, a.k, kBK, kTW);
  if (e == cudaSuccess)
    e = a.gain != nullptr && t.norm == 0 ? encode_rows_sw128(&tm_x, a.xhat, a.k, a.rows, a.k, kBK, t.bn)
                                         : encode_rows_sw128(&tm_x, a.x, a.k, a.rows, a.x_stride, kBK, t.bn);
  if (e != cudaSuccess) return e;
  // (the same for every call: the limit is the kernel's, and another thread may set it between this line and the launch)
  e = cudaFuncSetAttribute(linear_rows_kernel<ACT, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmemMost);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.wide + kTW - 1) / kTW) * t.xt * t.split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = t.smem;
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

template <int ACT, bool GATED>
cudaError_t launch_tiles(const LinearArgs& a, int bn, int num_sms, cudaStream_t stream) {
  TilesPlan t;
  t.bn = bn;
  t.boxes = (a.k + kBK - 1) / kBK;
  t.wt = (a.wide + bn - 1) / bn;
  t.xt = (a.rows + kPairRows - 1) / kPairRows;
  t.pairs = num_sms / 2;
  if (t.pairs > t.wt * t.xt) t.pairs = t.wt * t.xt;
  t.band = t.xt < 8 ? t.xt : 8;
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
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_tiles_kernel<ACT, GATED>, tm_w, tm_x, a, t);
}

// ------------------------------------------------------------ which kernel, which tiles
struct Choice {
  bool tiles;   // linear_tiles_kernel, else linear_rows_kernel
  int bn;       // rows of W, or of x, to a tile
  int split;    // CTAs that share a tile's K
  bool norm;    // the rows are normed inside the kernel
};

constexpr int kNormBytes = 40 * 1024;  // of shared memory that rows normed inside may take

// Whether rows_plan's CTAs norm their rows themselves: rows of a warp's lanes at most, done in two rounds, while the first
// boxes of W come.  That is a launch less, 2 us on the host; on the GPU 32 rows of 256 x 768 took 4.6 us for 4.7 with the
// norm's kernel in front, 8 of 1024 x 4096 7.6 for 7.9, 16 of 512 x 2048 5.9 for 5.6; by two warps a row 3 rows of 2048 x 12288
// took 16.3 for 15.1, so that they have the kernel.
bool norm_inside(const LinearArgs& a, int bn, int split) {
  const int lanes = norm_lanes(a.k), boxes = (a.k + kBK - 1) / kBK;
  return a.gain != nullptr && lanes <= 32 && (bn < a.rows ? bn : a.rows) * lanes <= 2 * kNormThreadsInside &&
         (boxes + split - 1) / split * bn * kBK * 2 <= kNormBytes;
}

// What each kernel takes, in us: fitted to 230 shapes (1 to 2048 rows, K 256 to 12288, 256 to 24576 rows of W) with every
// tile and split, where the choice was within 2% of the best on average and 32% at worst, and to a dozen with other ways to
// y.  A box of 64 columns costs a CTA the longer of the MMAs' own pace, its bytes' way from L2, shared with the other CTAs,
// and the ring's latency.  (512 rows of 4096 x 4096: 23 us on pairs of 128 rows of W, 36 on 128 x 128 tiles; 64 rows: 11.7
// with K cut in eight, 24 uncut; 777 x 1000 x 1003: 11.0 as 64-row tiles, 46 on 256 x 256 ones.)
float rows_us(const LinearArgs& a, int bn, int split, int num_sms) {
  const RowsPlan t = rows_plan(a, bn, split, false);
  const int wt = (a.wide + kTW - 1) / kTW;
  const int64_t ctas = static_cast<int64_t>(wt) * t.xt * split;
  const int64_t waves = (ctas + 2 * num_sms - 1) / (2 * num_sms) + (split > 4 && ctas > 9 * num_sms / 5 ? 1 : 0);
  const float kb = 16.f + bn / 8.f;
  const float box = fmaxf(fmaxf(0.29f, 0.99f / t.stages), kb * 0.0082f * (ctas > num_sms ? 2 : 1));
  const float col = 0.033f + (a.residual != nullptr ? 0.015f : 0.f) + (a.act == kActGelu ? 0.02f : a.act != kActNone ? 0.01f : 0.f);
  const float one = (t.boxes + split - 1) / split * box + 0.38f + (split > 1 ? 0.46f + (0.035f + 0.3f * col) * bn : col * bn);
  const float dram = static_cast<float>(a.wide) * a.k * 2.f / 6.7e6f + (split > 1 ? 0.46f : 0.f);
  return 2.2f + fmaxf(waves * one, dram) + 0.05f * fminf(waves * one, dram);
}

float tiles_us(const LinearArgs& a, int bn, int num_sms) {
  const int boxes = (a.k + kBK - 1) / kBK, pairs = num_sms / 2;
  const int64_t tiles = (static_cast<int64_t>(a.wide) + bn - 1) / bn * ((a.rows + kPairRows - 1) / kPairRows);
  const int64_t waves = (tiles + pairs - 1) / pairs;
  const float busy = tiles < pairs ? static_cast<float>(tiles) / pairs : 1.f;
  const float box = fmaxf(0.287f, (32.f + bn / 4.f) * busy * 0.00307f);
  // making y of a tile, in us for 256 columns: less where it is hidden behind the next tile's MMAs
  const bool apart = !rows16(a.y, a.y_stride);
  const float out = 2.6f + (apart ? 2.2f : 0.f) + (a.residual != nullptr ? 1.7f : 0.f) + (a.bias != nullptr ? 0.8f : 0.f) +
                    (a.act == kActGelu ? 2.2f : a.act != kActNone ? 1.2f : 0.f);
  const float mma = boxes * box, last = 1.5f + (out - 1.5f) * bn / 256;
  const float work = (waves - 1) * fmaxf(mma, last) + mma + last;
  const float dram = static_cast<float>(a.wide) * a.k * 2.f / 6.7e6f;
  return 3.2f + fmaxf(work, dram) + 0.05f * fminf(work, dram);
}

Choice choose(const LinearArgs& a, int num_sms) {
  Choice best = {};
  float least = INFINITY;
  for (int bn = 64; bn <= 256; bn += 32) {
    const float us = tiles_us(a, bn, num_sms);
    if (us < least) {
      least = us;
      best = {true, bn, 1, false};
    }
  }
  int last = 0;
  for (int most : {128, 96, 64, 48, 32, 16}) {
    const int xt = (a.rows + most - 1) / most, bn = ((a.rows + xt - 1) / xt + 15) / 16 * 16;
    if (bn == last) continue;
    last = bn;
    // (of many CTAs the pairs' tiles are always the better ones)
    if (static_cast<int64_t>((a.wide + kTW - 1) / kTW) * xt > 4 * num_sms) continue;
    for (int split : {1, 2, 3, 4, 5, 8}) {
      if (split > (a.k + kBK - 1) / kBK) break;
      const float us = rows_us(a, bn, split, num_sms);
      if (us < least) {
        least = us;
        best = {false, bn, split, norm_inside(a, bn, split)};
      }
    }
  }
  return best;
}

template <int ACT, bool GATED>
cudaError_t launch_product(const LinearArgs& a, const Choice& c, int num_sms, cudaStream_t stream) {
  return c.tiles ? launch_tiles<ACT, GATED>(a, c.bn, num_sms, stream)
                 : launch_rows<ACT, GATED>(a, rows_plan(a, c.bn, c.split, c.norm), stream);
}

template <int ACT>
cudaError_t launch_act(const LinearArgs& a, const Choice& c, int num_sms, cudaStream_t stream) {
  return a.gated ? launch_product<ACT, true>(a, c, num_sms, stream) : launch_product<ACT, false>(a, c, num_sms, stream);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  if (a.rows <= 0) return cudaSuccess;
  // One or two rows: W streamed past registers (4096 x 6144, one row 9.2 us for 11.6 as the tensor cores' N, normed 10.6 for
  // 12.9, two 10.5 and 12.5 for 11.7 and 14.2; 256 x 768 normed 2.0 and 2.4 for 4.4 and 4.2; 12288 x 4096, one row 16.9 for
  // 19.5.  Two rows of 11008 x 4096 took 18.6 for 17.8, four of 4096 x 6144 11.8 to 15.8 for 11.7 to 14.2.)
  if (a.rows <= few_rows(a.k)) return launch_linear_few(a, num_sms, stream);
  const Choice c = choose(a, num_sms);
  if (a.gain != nullptr && !c.norm) {
    // (all of a row in registers: 4000 rows of 920 take 4.8 us by warps, 8.0 by four of them; of 2976 11.7 by four, 16.5 by eight)
    const int team = a.k <= 1024 ? 32 : a.k <= 4096 ? 128 : kNormThreads, per_cta = kNormThreads / team;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.rows + per_cta - 1) / per_cta);
    cfg.blockDim = dim3(kNormThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, team == 32    ? linear_norm_kernel<32>
                                                   : team == 128 ? linear_norm_kernel<128>
                                                                 : linear_norm_kernel<kNormThreads>, a);
    if (e != cudaSuccess) return e;
  }
  switch (a.act) {
    case kActSilu:
      return launch_act<kActSilu>(a, c, num_sms, stream);
    case kActGelu:
      return launch_act<kActGelu>(a, c, num_sms, stream);
    case kActGeluTanh:
      return launch_act<kActGeluTanh>(a, c, num_sms, stream);
    default:
      return launch_act<kActNone>(a, c, num_sms, stream);
  }
}

}  // namespace dllm
