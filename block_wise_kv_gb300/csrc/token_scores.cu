// token_scores.cu — what a sampler reads off each row of logits, in one pass (sm_103a): with
// x the row, M its largest value and c the scale,
//   s = sum e^(c (x - M)),  a = sum e^(c (x - M)) c (x - M)
//   lse = c M + log s,  entropy = log s - a / s,  log p(t) = c (x_t - M) - log s,
// and the top_k largest with the lowest index first among equals.
//
// A CTA takes a row.  A thread takes 16-byte pieces of it, a CTA's width apart, and keeps the
// running (M, s, a) (references raised a batch of pieces at a time) and, for the alternatives,
// its largest value with the first piece that holds it.  These pairs are all different, and
// each stands for an element, so the top_k-th largest pair T is a bound: an element below it
// (smaller, or equal and in a later piece) has top_k others before it.  Only threads whose own
// pair is T or above hold elements at or above it, top_k of them: their pieces alone are read
// again, and what passes T, hardly more than top_k values, is ranked.
#include <math.h>

#include "layer_ops.cuh"
#include "sm103.cuh"

namespace dllm {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 512;        // elements ranked at once
constexpr float kFloor = -1000.f; // log2 of a weight that is zero: keeps 0 * -inf out of the sums

template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}

// Unsigned numbers in the order of the floats (+0 and -0 alike); 0 is below every one of them.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

struct Stat {
  float m, s, a;  // largest, sum of weights, sum of weight x log2 weight, relative to max(m, -FLT_MAX)
};
__device__ __forceinline__ float reference(float m) { return fmaxf(m, -3.402823466e38f); }

__device__ __forceinline__ Stat join(const Stat& x, const Stat& y, float c) {
  Stat z;
  z.m = fmaxf(x.m, y.m);
  const float r = reference(z.m);
  const float dx = fmaxf((reference(x.m) - r) * c, kFloor), dy = fmaxf((reference(y.m) - r) * c, kFloor);
  const float fx = ex2(dx), fy = ex2(dy);
  z.s = fx * x.s + fy * y.s;
  z.a = fx * (x.a + x.s * dx) + fy * (y.a + y.s * dy);
  return z;
}

// A row's pieces: piece v holds the elements at 16-byte boundary v of the row's memory, the first and the
// last possibly fewer than N of them.  Values that are not the row's read -inf.
template <typename T>
struct Row {
  const T* p;  // element 0
  int lead;    // places of piece 0 before it
  int n, pieces;
  __device__ __forceinline__ Row(const T* p_, int n_) : p(p_), n(n_) {
    lead = static_cast<int>((reinterpret_cast<uintptr_t>(p_) & 15) / sizeof(T));
    pieces = (lead + n + Piece<T>::N - 1) / Piece<T>::N;
  }
  __device__ __forceinline__ int first(int v) const { return v * Piece<T>::N - lead; }  // element of its place 0
  __device__ __forceinline__ bool whole(int v) const { return first(v) >= 0 && first(v) + Piece<T>::N <= n; }
  __device__ __forceinline__ void get(int v, float (&x)[Piece<T>::N]) const {
    const int e = first(v);
    if (whole(v)) {
      Piece<T>::get(__ldg(reinterpret_cast<const uint4*>(p + e)), x);
    } else {
#pragma unroll
      for (int i = 0; i < Piece<T>::N; ++i) x[i] = e + i >= 0 && e + i < n ? Piece<T>::one(p + e + i) : -INFINITY;
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) token_scores_kernel(const ScoreArgs a) {
  constexpr int N = Piece<T>::N;
  __shared__ Stat stats[kWarps];
  __shared__ uint64_t keys[kThreads];
  __shared__ uint64_t list[kList];
  __shared__ uint64_t bound_sh, prev_sh, round_sh[kWarps];
  __shared__ int owners[kMaxTop], n_owners, n_list;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float c = a.scale * 1.4426950408889634f;
  griddep_wait();
  griddep_launch_dependents();

  for (int j = blockIdx.x; j < a.rows; j += gridDim.x) {
    const Row<T> row(static_cast<const T*>(a.logits) + j * a.stride, a.vocab);
    // ---- statistics and this thread's largest
    Stat t = {-INFINITY, 0.f, 0.f};
    uint64_t best = 0;
    for (int v = tid; v < row.pieces; v += kThreads) {
      float x[N];
      row.get(v, x);
      float m = x[0];
#pragma unroll
      for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
      const uint64_t key = m > -INFINITY ? static_cast<uint64_t>(ordered(m)) << 32 | (0xFFFFFFFFu - v) : 0;
      best = key > best ? key : best;
      const float now = fmaxf(t.m, m), r = reference(now);
      const float d = fmaxf((reference(t.m) - r) * c, kFloor), f = ex2(d);
      t.a = f * (t.a + t.s * d);
      t.s *= f;
      t.m = now;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float u = max_nan((x[i] - r) * c, kFloor), e = ex2(u);
        t.s += e;
        t.a = fmaf(e, u, t.a);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Stat y = {__shfl_xor_sync(0xffffffffu, t.m, o), __shfl_xor_sync(0xffffffffu, t.s, o),
                      __shfl_xor_sync(0xffffffffu, t.a, o)};
      t = (lane & o) ? join(y, t, c) : join(t, y, c);
    }
    if (lane == 0) stats[warp] = t;
    keys[tid] = best;
    if (tid == 0) n_owners = n_list = 0;
    __syncthreads();
    t = stats[0];
    for (int w = 1; w < kWarps; ++w) t = join(t, stats[w], c);
    const bool bad = !(t.s < INFINITY) || t.m == INFINITY;  // a NaN or +inf
    const bool empty = !bad && t.m == -INFINITY;
    const float log_s = logf(t.s);
    if (tid == 0) {
      const float nan = __int_as_float(0x7FFFFFFF);
      if (bad) report_error(a.err, kErrRange);
      if (a.lse != nullptr) a.lse[j] = bad ? nan : empty ? -INFINITY : fmaf(t.m, a.scale, log_s);
      if (a.entropy != nullptr) a.entropy[j] = bad ? nan : empty ? 0.f : log_s - t.a / t.s * 0.6931471805599453f;
      if (a.tokens != nullptr) {
        const int tok = a.tokens[j];
        float lp = 0.f;
        if (bad) {
          lp = nan;
        } else if (tok >= a.vocab) {
          lp = nan;
          report_error(a.err, kErrBadShape);
        } else if (tok >= 0) {
          lp = empty ? -INFINITY : (Piece<T>::one(row.p + tok) - t.m) * a.scale - log_s;
        }
        a.logp[j] = lp;
      }
    }
    // ---- the alternatives
    if (a.top > 0) {
      int* ids = a.top_ids + static_cast<int64_t>(j) * a.top;
      float* lps = a.top_logp + static_cast<int64_t>(j) * a.top;
      if (bad || empty) {
        if (tid < a.top) {
          ids[tid] = -1;
          lps[tid] = bad ? __int_as_float(0x7FFFFFFF) : -INFINITY;
        }
      } else {
        int before = 0;  // threads whose pair is larger
        if (best != 0)
          for (int i = 0; i < kThreads; ++i) before += keys[i] > best;
        if (best != 0 && before < a.top) owners[atomicAdd(&n_owners, 1)] = tid;
        if (tid == 0) bound_sh = 0;
        __syncthreads();
        if (best != 0 && before == a.top - 1) bound_sh = best;  // none where fewer threads hold anything
        __syncthreads();
        const uint64_t bound = bound_sh;
        const int no = n_owners, each = (row.pieces + kThreads - 1) / kThreads;
        for (int i = tid; i < no * each; i += kThreads) {
          const int v = owners[i % no] + i / no * kThreads;
          if (v >= row.pieces) continue;
          float x[N];
          row.get(v, x);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            if (!(x[e] > -INFINITY)) continue;
            const uint64_t value = static_cast<uint64_t>(ordered(x[e])) << 32;
            if ((value | (0xFFFFFFFFu - v)) < bound) continue;
            const int at = atomicAdd(&n_list, 1);
            if (at < kList) list[at] = value | (0xFFFFFFFFu - (row.first(v) + e));
          }
        }
        __syncthreads();
        const int nl = n_list;
        if (nl <= kList) {
          for (int i = tid; i < nl; i += kThreads) {
            int rank = 0;
            for (int o = 0; o < nl; ++o) rank += list[o] > list[i];
            if (rank < a.top) {
              ids[rank] = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(list[i]));
              lps[rank] = (unordered(static_cast<uint32_t>(list[i] >> 32)) - t.m) * a.scale - log_s;
            }
          }
          for (int i = nl + tid; i < a.top; i += kThreads) {
            ids[i] = -1;
            lps[i] = -INFINITY;
          }
        } else {  // so many in so few threads' pieces: one after the other
          if (tid == 0) prev_sh = ~0ull;
          __syncthreads();
          for (int rank = 0; rank < a.top; ++rank) {  // (there are more than kList of them)
            const uint64_t prev = prev_sh;
            uint64_t most = 0;
            for (int i = tid; i < no * each; i += kThreads) {
              const int v = owners[i % no] + i / no * kThreads;
              if (v >= row.pieces) continue;
              float x[N];
              row.get(v, x);
#pragma unroll
              for (int e = 0; e < N; ++e) {
                const uint64_t key =
                    x[e] > -INFINITY
                        ? static_cast<uint64_t>(ordered(x[e])) << 32 | (0xFFFFFFFFu - (row.first(v) + e))
                        : 0;
                if (key < prev && key > most) most = key;
              }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
              const uint64_t y = __shfl_xor_sync(0xffffffffu, most, o);
              most = y > most ? y : most;
            }
            if (lane == 0) round_sh[warp] = most;
            __syncthreads();
            if (tid == 0) {
              for (int w = 1; w < kWarps; ++w) most = round_sh[w] > most ? round_sh[w] : most;
              prev_sh = most;
              ids[rank] = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(most));
              lps[rank] = (unordered(static_cast<uint32_t>(most >> 32)) - t.m) * a.scale - log_s;
            }
            __syncthreads();
          }
        }
      }
    }
    __syncthreads();  // the next row's
  }
}

}  // namespace

cudaError_t launch_token_scores(const ScoreArgs& a, int num_sms, cudaStream_t stream) {
  if (a.rows <= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.rows < 4 * num_sms ? a.rows : 4 * num_sms);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.fp32 ? cudaLaunchKernelEx(&cfg, token_scores_kernel<float>, a)
                : cudaLaunchKernelEx(&cfg, token_scores_kernel<__nv_bfloat16>, a);
}

}  // namespace dllm
