// kv8_write.cu — rows of K and V into the 8-bit paged cache.
//
// A group is 16 token positions of one head: amax over its new rows gives the
// scale s = 2^e, the smallest power of two with amax <= 448 s (-60 <= e <= 60),
// and code = e4m3(x / s).  x / s is exact (a power of two), so the only rounding
// is the one to e4m3.  Where rows of the group stay, s is at least their present
// scale and their codes are multiplied by the ratio, again a power of two: exact
// unless the result is an e4m3 subnormal.  A scale of amax / 448 would fill the
// last bit of the range, but every growth would round all kept rows again.
//
// Bound: HBM, 3 bytes a value (read 2, write 1).  A warp takes one group of K or of V:
// 16 rows of 256 bytes, every load in flight before the first is used, 8-byte code
// stores.  Groups start where a block starts or where a position is a multiple of 16, so
// a CTA takes a slice of packed rows, finds the groups that begin in it, and deals (group,
// head) items to its warps.
//
// Measured (d = 128): four whole sequences of 5120 rows of 32 heads from the bf16 pools
// 74.8 us, 6.7 TB/s, a copy's rate (118 us with fp32 maxima and products one by one and
// the rare values in the same registers), and out of packed rows 77.2 us, 6.5 TB/s.  512
// block rows of 32 heads 5.7 us, 128 single tokens of 8 heads 4.4 us: a launch and the dependent trips cu_block -> lengths -> page
// -> rows, scale.
#include <algorithm>

#include "attn_common.cuh"
#include "kv8.cuh"

namespace dllm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;
constexpr int kMaxSlice = 32;  // packed rows a CTA looks at, at most
constexpr int kCuInSmem = 1024;  // batches up to this many sequences are searched in shared memory

struct Group {
  int row;      // first new row (packed)
  int t0, n;    // new rows are slots t0 .. t0 + n of the group
  int keep_lo;  // rows that stay: slots 0 .. keep_lo, and t0 + n .. keep_hi
  int keep_hi;
  int page, quarter;
};

// The smallest e in [-60, 60] with amax <= 448 * 2^e, for the magnitude bits of a finite bf16.
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  // 448 = 1.75 * 2^8; 1.75 is mantissa 96 of 128
  const int e = static_cast<int>(amax_bits >> 7) - 127 - ((amax_bits & 127u) <= 96u ? 8 : 7);
  return min(max(e, -kKv8MaxExp), kKv8MaxExp);
}
__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ float2 bf16x2_f32(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// Two e4m3 codes to fp32 (exact).
__device__ __forceinline__ float2 e4m3x2_f32(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
// Non-finite values of a bf16 pair to not-a-number (so that they become e4m3's).
__device__ __forceinline__ uint32_t only_nan(uint32_t u) {
  if ((u & 0x7f80u) == 0x7f80u) u |= 0x7fu;
  if ((u & 0x7f800000u) == 0x7f800000u) u |= 0x7f0000u;
  return u;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Eight codes of eight bf16 values x / s (s a power of two, inv = 1 / s: exact products).
__device__ __forceinline__ uint2 codes_of(const uint4& x, uint64_t inv2) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint16_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(w[k] << 16), "r"(w[k] & 0xffff0000u));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(v), "l"(inv2));
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
    c[k] = cvt_e4m3x2(lo, hi);
  }
  return make_uint2(c[0] | (static_cast<uint32_t>(c[1]) << 16), c[2] | (static_cast<uint32_t>(c[3]) << 16));
}

// The group of one pool: the lane's pieces x[i] are rows kRows * i + lane / kLanes, 8 columns from 8 * (lane % kLanes).
// Groups with nothing out of the ordinary take the short way; what is rare is kept out of its registers and reads the
// rows again from src (row t of the group at src + t * row, at this lane's columns).
template <int D>
__device__ __forceinline__ void quantise(const uint4 (&x)[D / 16], const __nv_bfloat16* src, int64_t row, const Group& g,
                                         uint8_t* codes, float* scale, int lane, int& err) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIter = 16 / kRows;
  const int sub = lane / kLanes, col = (lane % kLanes) * 8;
  uint8_t* const mine = codes + sub * D + col;  // row sub; row kRows * i + sub is kRows * D * i further
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kIter; ++i)
    m = max_u16x2(m, max_u16x2(max_u16x2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                               max_u16x2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
  uint32_t amax = max(m & 0xffffu, m >> 16);
  const bool odd = amax >= 0x7f80u;
  if (odd) {  // a value that is not finite takes no part in the scale
    err |= kErrRange;
    amax = 0;
#pragma unroll 1
    for (int t = sub; t < 16; t += kRows) {
      if (t < g.t0 || t >= g.t0 + g.n) continue;
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        const uint32_t v = __ldg(reinterpret_cast<const uint16_t*>(src + t * row) + k) & 0x7fffu;
        if (v < 0x7f80u) amax = max(amax, v);
      }
    }
    __syncwarp();
    amax = __reduce_max_sync(0xffffffffu, amax);
  }
  if (amax > (static_cast<uint32_t>(127 + 8 + kKv8MaxExp) << 7) + 96u) err |= kErrRange;  // beyond 448 * 2^60
  float s = two_to(scale_exponent(amax));
  const bool keeps = g.keep_lo > 0 || g.keep_hi > g.t0 + g.n;
  if (keeps) {
    const float old = *scale;
    if (old > s) {
      s = old;
    } else if (old < s) {
      const float ratio = __fdiv_rn(old, s);
#pragma unroll 1
      for (int i = 0; i < kIter; ++i) {
        const int t = i * kRows + sub;
        if (t < g.keep_lo || (t >= g.t0 + g.n && t < g.keep_hi)) {
          uint2* p = reinterpret_cast<uint2*>(mine + i * kRows * D);
          const uint2 c = *p;
          uint32_t out[2];
          const uint32_t in[2] = {c.x, c.y};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 lo = e4m3x2_f32(static_cast<uint16_t>(in[k])), hi = e4m3x2_f32(static_cast<uint16_t>(in[k] >> 16));
            out[k] = static_cast<uint32_t>(cvt_e4m3x2(lo.x * ratio, lo.y * ratio)) |
                     (static_cast<uint32_t>(cvt_e4m3x2(hi.x * ratio, hi.y * ratio)) << 16);
          }
          *p = make_uint2(out[0], out[1]);
        }
      }
    }
  }
  const bool exact = (__float_as_uint(s) & 0x7fffffu) == 0;  // else a present scale of another kind: divided by
  if (exact && !odd) {
    const float inv = __frcp_rn(s);
    uint64_t inv2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(inv2) : "f"(inv));
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int t = i * kRows + sub;
      const uint2 c = codes_of(x[i], inv2);
      if (t >= g.t0 && t < g.t0 + g.n) *reinterpret_cast<uint2*>(mine + i * kRows * D) = c;
    }
  } else {
#pragma unroll 1
    for (int t = sub; t < 16; t += kRows) {
      if (t < g.t0 || t >= g.t0 + g.n) continue;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {  // a pair of values at a time
        const float2 f = bf16x2_f32(only_nan(__ldg(reinterpret_cast<const uint32_t*>(src + t * row) + k)));
        *reinterpret_cast<uint16_t*>(codes + t * D + col + 2 * k) = cvt_e4m3x2(__fdiv_rn(f.x, s), __fdiv_rn(f.y, s));
      }
    }
  }
  __syncwarp();  // every lane has read the old scale
  if (lane == 0) *scale = s;
}

template <int D, bool POOL>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv8_write_kernel(const Kv8WriteArgs a, int slice, int heads_per_cta) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIter = 16 / kRows;
  __shared__ int cu[kCuInSmem + 1];
  __shared__ Group groups[kMaxSlice];
  __shared__ int n_groups;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const BatchArgs& bt = a.bt;
  const int row0 = blockIdx.x * slice;
  const bool in_smem = bt.batch <= kCuInSmem;
  int err = 0;
  griddep_wait();
  griddep_launch_dependents();
  if (t == 0) n_groups = 0;
  // One CTA compares all blocks with the sums: one that they leave no rows is met by no search below.
  const bool looks = blockIdx.x == 0 && blockIdx.y == 0;
  auto rows_of = [&](int b) { return __ldg(bt.seq_len + b) == 0 ? 0 : __ldg(bt.block_len + b); };  // (a place without a request)
  const int rows_t = looks && t < bt.batch ? rows_of(t) : 0;
  if (in_smem)
    for (int i = t; i <= bt.batch; i += kThreads) cu[i] = __ldg(bt.cu_block + i);
  __syncthreads();
  const int* cub = in_smem ? cu : bt.cu_block;
  for (int b = t; looks && b < bt.batch; b += kThreads)
    if (cub[b + 1] - cub[b] != (b == t ? rows_t : rows_of(b))) err |= kErrBadShape;
  const int total = min(cub[bt.batch], bt.total_block_rows);
  if (row0 == 0 && t == 0 && (cub[bt.batch] < 0 || cub[bt.batch] > bt.total_block_rows)) err |= kErrBadShape;
  if (row0 >= total) {
    if (err) report_error(bt.err, err);
    return;
  }
  if (t < slice && row0 + t < total) {
    const int j = row0 + t;
    int lo = 0, hi = bt.batch;  // the last sequence that starts at or before row j
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cub[mid] <= j)
        lo = mid;
      else
        hi = mid;
    }
    const int b = lo, first_row = cub[b], next_row = cub[b + 1], i = j - first_row;
    const int n = __ldg(bt.seq_len + b), s = __ldg(bt.block_start + b), len = __ldg(bt.block_len + b);
    const int pos = s + i;
    // The whole block lies in its own packed rows and within the bound: a group below reads up to 16 of them from row j on.
    if (first_row < 0 || next_row < first_row || len > min(next_row, bt.total_block_rows) - first_row || n < 0 ||
        n > bt.max_seq_len || s < 0 || len < 0 || len > n - s || i < 0 || i >= len || pos / kPage >= bt.max_pages) {
      err |= kErrBadShape;
    } else if (i == 0 || pos % kKv8Group == 0) {
      const int pg = __ldg(bt.block_table + static_cast<size_t>(b) * bt.max_pages + pos / kPage);
      if (pg < 0 || pg >= bt.num_pages) {
        err |= kErrBadPage;
      } else {
        Group g;
        const int first = pos / kKv8Group * kKv8Group;
        g.row = j;
        g.t0 = pos - first;
        g.n = min(kKv8Group - g.t0, len - i);
        g.keep_lo = g.t0;
        g.keep_hi = min(kKv8Group, n - first);
        g.page = pg;
        g.quarter = (first % kPage) / kKv8Group;
        groups[atomicAdd(&n_groups, 1)] = g;
      }
    }
  }
  __syncthreads();
  // an item is a group of one head's K or V
  const int h0 = blockIdx.y * heads_per_cta, nh = min(heads_per_cta, a.kv.n_kv_heads - h0);
  const int items = n_groups * nh * 2;
  const int sub = lane / kLanes, col = (lane % kLanes) * 8;
  for (int it = warp; it < items; it += kWarps) {
    const bool is_k = (it & 1) == 0;
    const Group g = groups[(it >> 1) / nh];
    const int h = h0 + (it >> 1) % nh;
    const size_t unit = static_cast<size_t>(g.page) * a.kv.n_kv_heads + h, slot = unit * kPage + g.quarter * kKv8Group;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_k ? a.k_src : a.v_src) + col;
    int64_t row = D;
    if (POOL) {
      src += slot * D;
    } else {
      row = is_k ? a.k_row : a.v_row;
      src += (g.row - g.t0) * row + h * (is_k ? a.k_head : a.v_head);
    }
    uint4 x[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int tt = i * kRows + sub;
      x[i] = tt >= g.t0 && tt < g.t0 + g.n ? __ldg(reinterpret_cast<const uint4*>(src + tt * row)) : make_uint4(0, 0, 0, 0);
    }
    quantise<D>(x, src, row, g, (is_k ? a.kv.k : a.kv.v) + slot * D, (is_k ? a.kv.k_scale : a.kv.v_scale) + unit * kKv8Groups + g.quarter,
                lane, err);
  }
  if (err) report_error(bt.err, err);
}

}  // namespace

cudaError_t launch_kv8_write(const Kv8WriteArgs& a, int num_sms, cudaStream_t stream) {
  const int rows = a.bt.total_block_rows, heads = a.kv.n_kv_heads;
  // Rows to a group, by the mean block: single tokens make every row a group of its own.
  const int mean = std::min(kKv8Group, std::max(1, rows / a.bt.batch));
  const long long items = 2ll * heads * ((rows + mean - 1) / mean), resident = static_cast<long long>(kCtasPerSm) * num_sms;
  int slice, hc;
  // Enough for every resident warp several times over: wide slices, whose search serves more items (whole sequences 74.8
  // us; 75.6 with narrow ones).  Else latency: about an item to a warp (single tokens 4.4 us, blocks 5.7; 42.0 and 6.2
  // with the wide ones).
  if (items >= 4 * kWarps * resident) {
    slice = kMaxSlice;
    hc = 4;
  } else {
    slice = std::min(16, 4 * mean);
    hc = std::max(1, kWarps * mean / (2 * slice));
  }
  hc = std::min(hc, heads);
  const dim3 grid((rows + slice - 1) / slice, (heads + hc - 1) / hc);
  if (a.head_dim == 128)
    return a.from_pool ? attn::launch_pdl(kv8_write_kernel<128, true>, grid, kThreads, 0, 0, stream, a, slice, hc)
                       : attn::launch_pdl(kv8_write_kernel<128, false>, grid, kThreads, 0, 0, stream, a, slice, hc);
  return a.from_pool ? attn::launch_pdl(kv8_write_kernel<64, true>, grid, kThreads, 0, 0, stream, a, slice, hc)
                     : attn::launch_pdl(kv8_write_kernel<64, false>, grid, kThreads, 0, 0, stream, a, slice, hc);
}

}  // namespace dllm
