// token_scores.cu — what a sampler reads off each row of logits, in one pass (sm_103a): with
// x the row, M its largest value and c the scale,
//   s = sum e^(c (x - M)),  a = sum e^(c (x - M)) c (x - M)
//   lse = c M + log s,  entropy = log s - a / s,  log p(t) = c (x_t - M) - log s,
// and the top_k largest with the lowest index first among equals.
//
// A CTA takes a row, or where rows are few a cluster of up to eight does: each CTA every
// eighth stretch of the row, and the first one joins what they leave in its shared memory.
// A thread takes 16-byte pieces, a stretch apart, four at a time, and keeps its running
// (reference, s, a), raised once a batch.  Exponents are powers of two: u = x c log2 e - R is
// one FMA from the reference R, two elements to an instruction.
//
// For the alternatives a thread keeps its largest value with the first piece that holds it.
// These pairs are all different, and each stands for an element, so a value that top_k of
// them reach is a bound: an element below it (smaller, or equal and in a later piece) has
// top_k others before it.  The bound is the top_k-th largest of the pairs of 64 groups of
// four threads; only threads whose own pair is at or above it hold such elements, hardly
// more than top_k of them: their pieces alone are read again, and what passes is ranked.
#include <math.h>

#include "layer_ops.cuh"
#include "sm103.cuh"

namespace dllm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;          // pieces a thread has on their way
constexpr int kMaxCluster = 8;
constexpr int kGroups = kThreads / 4;
constexpr int kOwners = 4 * kMaxTop;  // threads that can reach the bound
constexpr int kList = 512;         // elements ranked at once
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The fast form takes what lies below kLow for kLow, which as a power of two times c log2 e is exact, so that masked logits
// bring no infinity up.  Its weight is zero all the same beside a largest logit in +-kFar, at a scale in [kLeast, kMost] (in
// powers of two).  Other rows take the slow form.
constexpr float kLow = -32768.f, kFar = 16384.f, kLeast = 1.f / 64, kMost = 64.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) { return log2f(x); }

// Two floats to an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t x, uint32_t y) {
  uint32_t z;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
  return z;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t x, uint32_t y) {
  uint32_t z;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
  return z;
}
__device__ __forceinline__ float2 unpack(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// A 16-byte piece: N values; its largest (a NaN only where there is nothing else); its pairs, none below kLow.
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
  static __device__ __forceinline__ float largest(const uint4& u) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  static __device__ __forceinline__ void pairs(const uint4& u, float2 (&p)[2]) {
    p[0] = make_float2(max_nan(__uint_as_float(u.x), kLow), max_nan(__uint_as_float(u.y), kLow));
    p[1] = make_float2(max_nan(__uint_as_float(u.z), kLow), max_nan(__uint_as_float(u.w), kLow));
  }
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ uint32_t bits(const float* p) { return __float_as_uint(__ldg(p)); }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kLow2 = 0xC700C700u;  // kLow, twice
  static __device__ __forceinline__ void get(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ float largest(const uint4& u) {
    const float2 f = unpack(max_bf16x2(max_bf16x2(u.x, u.y), max_bf16x2(u.z, u.w)));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ void pairs(const uint4& u, float2 (&p)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = unpack(max_nan_bf16x2(w[i], kLow2));
  }
  static __device__ __forceinline__ uint32_t bits(const __nv_bfloat16* p) {
    return __ldg(reinterpret_cast<const unsigned short*>(p));
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __uint_as_float(bits(p) << 16); }
};

// Unsigned numbers in the order of the floats (+0 and -0 alike); 0 is below every one of them.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// A value and where it is, the larger first, of equal ones the one in front; 0: none.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t at) {
  return x > -INFINITY ? static_cast<uint64_t>(ordered(x)) << 32 | (0xFFFFFFFFu - at) : 0;
}
__device__ __forceinline__ float value_of(uint64_t key) { return unordered(static_cast<uint32_t>(key >> 32)); }
__device__ __forceinline__ int place_of(uint64_t key) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key)); }

// Sums of weights 2^(u - r) and of weight x (u - r), u = x c log2 e.  The slow form keeps r in units of x, and works on
// differences of x, which do not overflow.
template <bool SLOW>
struct Stat {
  float r, s, a;
  static __device__ __forceinline__ float apart(float x, float y, float c) { return SLOW ? fmaxf((x - y) * c, -1000.f) : x - y; }
  __device__ __forceinline__ void join(const Stat& y, float c) {
    const float n = fmaxf(r, y.r), dx = apart(r, n, c), dy = apart(y.r, n, c);
    const float fx = ex2(dx), fy = ex2(dy);
    a = fx * (a + s * dx) + fy * (y.a + y.s * dy);
    s = fx * s + fy * y.s;
    r = n;
  }
};

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
  __device__ __forceinline__ uint4 load(int v) const { return __ldg(reinterpret_cast<const uint4*>(p + first(v))); }
  __device__ __noinline__ uint4 edge(int v) const {
    constexpr int N = Piece<T>::N, W = 32 * 4 / N;
    uint32_t w[4] = {0, 0, 0, 0};
    const int e = first(v);
    for (int i = 0; i < N; ++i) {
      const uint32_t b = e + i >= 0 && e + i < n ? Piece<T>::bits(p + e + i) : sizeof(T) == 2 ? 0xFF80u : 0xFF800000u;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i * W / 32 == k) w[k] |= b << (i * W % 32);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 get(int v) const { return whole(v) ? load(v) : edge(v); }
};

// The slow form's sums of all pieces, by one CTA.
template <typename T>
__device__ __noinline__ Stat<true> slow_sums(const Row<T>& row, float c, int tid) {
  constexpr int N = Piece<T>::N;
  constexpr float kMin = -3.402823466e38f;
  Stat<true> t = {kMin, 0.f, 0.f};
  for (int v = tid; v < row.pieces; v += kThreads) {
    float x[N];
    Piece<T>::get(row.get(v), x);
    Stat<true> p = {kMin, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) p.r = fmaxf(p.r, x[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float u = max_nan((x[i] - p.r) * c, -1000.f), e = ex2(u);
      p.s += e;
      p.a = fmaf(e, u, p.a);
    }
    t.join(p, c);
  }
  return t;
}

// The sums of a CTA's threads, in a fixed order, to all of them.
template <bool SLOW>
__device__ __forceinline__ Stat<SLOW> block_join(Stat<SLOW> t, float c, float (*sh)[3], int tid) {
  const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat<SLOW> y = {__shfl_down_sync(0xffffffffu, t.r, o), __shfl_down_sync(0xffffffffu, t.s, o),
                    __shfl_down_sync(0xffffffffu, t.a, o)};
    t.join(y, c);
  }
  if (lane == 0) {
    sh[warp][0] = t.r;
    sh[warp][1] = t.s;
    sh[warp][2] = t.a;
  }
  __syncthreads();
  t = {sh[0][0], sh[0][1], sh[0][2]};
#pragma unroll 1
  for (int w = 1; w < kWarps; ++w) t.join({sh[w][0], sh[w][1], sh[w][2]}, c);
  return t;
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

struct Shared {
  float stat[kWarps][3];
  uint64_t group[kGroups];
  uint64_t list[kList];
  uint64_t best[kMaxTop];  // this CTA's alternatives, largest first
  uint64_t bound, prev, round[kWarps];
  int owners[kOwners], n_owners, n_list;
  // what the CTAs of a cluster leave with the first one
  float part[kMaxCluster][3];
  uint64_t part_key[kMaxCluster];
  uint64_t part_best[kMaxCluster * kMaxTop];
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) token_scores_kernel(const ScoreArgs a, int cluster) {
  constexpr int N = Piece<T>::N;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster > 1 ? static_cast<int>(blockIdx.x) % cluster : 0;
  const int stretch = kThreads * cluster;
  const float c = fminf(a.scale * kLog2e, 3.402823466e38f);
  griddep_wait();
  griddep_launch_dependents();

  for (int j = static_cast<int>(blockIdx.x) / cluster; j < a.rows; j += static_cast<int>(gridDim.x) / cluster) {
    const Row<T> row(static_cast<const T*>(a.logits) + j * a.stride, a.vocab);
    const int whole_from = row.lead > 0 ? 1 : 0, whole_to = (row.lead + row.n) / N;  // whole pieces
    // ---- sums, and this thread's largest
    float m = kLow, r = kLow * c, top = -INFINITY;
    int top_v = 0;
    float2 s2 = {0.f, 0.f}, a2 = {0.f, 0.f};
    for (int v0 = rank * kThreads + tid; v0 < row.pieces; v0 += kBatch * stretch) {
      uint4 q[kBatch];
      if (v0 >= whole_from && v0 + (kBatch - 1) * stretch < whole_to) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) q[b] = row.load(v0 + b * stretch);
      } else {
#pragma unroll 1
        for (int b = 0; b < kBatch; ++b) {
          const uint4 u = row.get(v0 + b * stretch);
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            if (k == b) q[k] = u;
        }
      }
      float most = m;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float l = Piece<T>::largest(q[b]);
        most = fmaxf(most, l);
        if (l > top) {
          top = l;
          top_v = v0 + b * stretch;
        }
      }
      const float now = most * c, d = r - now, f = ex2(d);
      a2 = fma2(s2, {d, d}, a2);
      a2 = fma2(a2, {f, f}, {0.f, 0.f});
      s2 = fma2(s2, {f, f}, {0.f, 0.f});
      m = most;
      r = now;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        float2 p[N / 2];
        Piece<T>::pairs(q[b], p);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float2 u = fma2(p[i], {c, c}, {-r, -r});
          const float2 e = {ex2(u.x), ex2(u.y)};
          s2 = add2(s2, e);
          a2 = fma2(e, u, a2);
        }
      }
    }
    const uint64_t best = key_of(top, top_v);
    Stat<false> t = {r, s2.x + s2.y, a2.x + a2.y};
    t = block_join(t, c, sh.stat, tid);

    // ---- this CTA's alternatives (the row's largest at least), as keys of element numbers
    const int want = a.top > 0 ? a.top : 1;
    {
      uint64_t g = best;
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        const uint64_t y = __shfl_xor_sync(0xffffffffu, g, o);
        g = y > g ? y : g;
      }
      if ((tid & 3) == 0) sh.group[tid >> 2] = g;
      if (tid == 0) {
        sh.bound = 0;
        sh.n_owners = sh.n_list = 0;
      }
      if (tid < kMaxTop) sh.best[tid] = 0;
      __syncthreads();
      if (tid < kGroups) {
        const uint64_t mine = sh.group[tid];
        int before = 0;
#pragma unroll 8
        for (int i = 0; i < kGroups; ++i) before += sh.group[i] > mine;
        if (mine != 0 && before == want - 1) sh.bound = mine;  // none where fewer hold anything
      }
      __syncthreads();
      const uint64_t bound = sh.bound;
      if (best != 0 && best >= bound) sh.owners[atomicAdd(&sh.n_owners, 1)] = tid;
      __syncthreads();
      const int no = sh.n_owners, each = (row.pieces + stretch - 1) / stretch;
      for (int i = tid; i < no * each; i += kThreads) {
        const int v = sh.owners[i % no] + rank * kThreads + i / no * stretch;
        if (v >= row.pieces) continue;
        float x[N];
        Piece<T>::get(row.get(v), x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (x[e] > -INFINITY && key_of(x[e], v) >= bound) {
            const int at = atomicAdd(&sh.n_list, 1);
            if (at < kList) sh.list[at] = key_of(x[e], row.first(v) + e);
          }
        }
      }
      __syncthreads();
      const int nl = sh.n_list;
      if (nl <= kList) {
        for (int i = tid; i < nl; i += kThreads) {
          int before = 0;
          for (int o = 0; o < nl; ++o) before += sh.list[o] > sh.list[i];
          if (before < want) sh.best[before] = sh.list[i];
        }
      } else {  // so many in so few threads' pieces: one after the other
        if (tid == 0) sh.prev = ~0ull;
        __syncthreads();
        for (int k = 0; k < want; ++k) {
          const uint64_t prev = sh.prev;
          uint64_t most = 0;
          for (int i = tid; i < no * each; i += kThreads) {
            const int v = sh.owners[i % no] + rank * kThreads + i / no * stretch;
            if (v >= row.pieces) continue;
            float x[N];
            Piece<T>::get(row.get(v), x);
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const uint64_t key = key_of(x[e], row.first(v) + e);
              if (key < prev && key > most) most = key;
            }
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const uint64_t y = __shfl_xor_sync(0xffffffffu, most, o);
            most = y > most ? y : most;
          }
          if (lane == 0) sh.round[warp] = most;
          __syncthreads();
          if (tid == 0) {
            for (int w = 1; w < kWarps; ++w) most = sh.round[w] > most ? sh.round[w] : most;
            sh.prev = sh.best[k] = most;
          }
          __syncthreads();
        }
      }
      __syncthreads();
    }

    // ---- the cluster's parts meet in its first CTA
    if (cluster > 1) {
      const uint32_t base = mapa_shared(smem_u32(&sh), 0) - smem_u32(&sh);
      if (tid == 0) {
        st_cluster_f32(base + smem_u32(&sh.part[rank][0]), t.r);
        st_cluster_f32(base + smem_u32(&sh.part[rank][1]), t.s);
        st_cluster_f32(base + smem_u32(&sh.part[rank][2]), t.a);
      }
      if (tid < want) st_cluster_u64(base + smem_u32(&sh.part_best[rank * want + tid]), sh.best[tid]);
      cluster_arrive_release();
      cluster_wait_acquire();
      if (rank == 0) {
        t = {sh.part[0][0], sh.part[0][1], sh.part[0][2]};
        for (int i = 1; i < cluster; ++i) t.join({sh.part[i][0], sh.part[i][1], sh.part[i][2]}, c);
        if (tid < kMaxTop) sh.best[tid] = 0;
        __syncthreads();
        if (tid < cluster * want) {
          const uint64_t mine = sh.part_best[tid];
          int before = 0;
          for (int i = 0; i < cluster * want; ++i) before += sh.part_best[i] > mine;
          if (mine != 0 && before < want) sh.best[before] = mine;
        }
        __syncthreads();
      }
    }

    // ---- results
    if (rank == 0) {
      const uint64_t first = sh.best[0];
      const float largest = first != 0 ? value_of(first) : -INFINITY;
      const bool slow = largest != INFINITY && (c < kLeast || c > kMost ||
                                                (first != 0 && (fabsf(largest) > kFar || fabsf(largest) * c > kFar)));
      float ref = t.r, s = t.s, wa = t.a;
      if (slow) {
        const Stat<true> z = block_join(slow_sums(row, c, tid), c, sh.stat, tid);
        ref = z.r;
        s = z.s;
        wa = z.a;
      }
      const bool bad = !(s < INFINITY) || largest == INFINITY;  // a NaN or +inf
      const bool empty = !bad && first == 0;
      const float nan = __int_as_float(0x7FFFFFFF), ls = lg2(s);
      // log of the sum relative to the largest; log p of a logit
      const float log_s = ((slow ? 0.f : fmaf(-largest, c, ref)) + ls) * kLn2;
      auto logp = [&](float x) { return fmaf(x - largest, a.scale, -log_s); };
      if (tid == 0) {
        if (bad) report_error(a.err, kErrRange);
        if (a.lse != nullptr)
          a.lse[j] = bad ? nan : empty ? -INFINITY : fmaf(largest, a.scale, log_s);
        if (a.entropy != nullptr) a.entropy[j] = bad ? nan : empty ? 0.f : (ls - wa / s) * kLn2;
      }
      if (tid == 32 && a.tokens != nullptr) {
        const int tok = a.tokens[j];
        float lp = 0.f;
        if (tok >= a.vocab) report_error(a.err, kErrBadShape);
        if (bad || tok >= a.vocab)
          lp = nan;
        else if (tok >= 0)
          lp = empty ? -INFINITY : logp(Piece<T>::one(row.p + tok));
        a.logp[j] = lp;
      }
      if (tid >= 64 && tid - 64 < a.top) {
        const uint64_t key = bad ? 0 : sh.best[tid - 64];
        const int64_t at = static_cast<int64_t>(j) * a.top + tid - 64;
        a.top_ids[at] = key != 0 ? place_of(key) : -1;
        a.top_logp[at] = bad ? nan : key != 0 ? logp(value_of(key)) : -INFINITY;
      }
    }
    __syncthreads();  // the next row's
    if (cluster > 1) {  // what the first CTA has of this row is read
      cluster_arrive_release();
      cluster_wait_acquire();
    }
  }
}

}  // namespace

cudaError_t launch_token_scores(const ScoreArgs& a, int num_sms, cudaStream_t stream) {
  if (a.rows <= 0) return cudaSuccess;
  // Few rows: a cluster to each, so that all of them fill the SMs, as long as a CTA has a batch of pieces for each thread.
  const int pieces = a.vocab / (a.fp32 ? 4 : 8);
  int cluster = 1;
  while (cluster < kMaxCluster && static_cast<int64_t>(a.rows) * cluster * 2 <= 4 * num_sms &&
         pieces >= cluster * 2 * kThreads * kBatch)
    cluster *= 2;
  const int most = 4 * num_sms / cluster;  // rows at once
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.rows < most ? a.rows : most) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return a.fp32 ? cudaLaunchKernelEx(&cfg, token_scores_kernel<float>, a, cluster)
                : cudaLaunchKernelEx(&cfg, token_scores_kernel<__nv_bfloat16>, a, cluster);
}

}  // namespace dllm
