// token_scores.cu — what a sampler reads off each row of logits, in one pass (sm_103a): with
// x the row, M its largest value and c the scale,
//   s = sum e^(c (x - M)),  a = sum e^(c (x - M)) c (x - M)
//   lse = c M + log s,  entropy = log s - a / s,  log p(t) = c (x_t - M) - log s,
// and the top_k largest with the lowest index first among equals.
//
// A team takes a row: a CTA, or where rows are many a warp, or where they are few a cluster
// of up to eight CTAs (each every eighth stretch of the row, the first one joins what they
// leave in its shared memory).  A thread takes 16-byte pieces, a stretch apart, four at a
// time with the next four on their way, and keeps its running (reference, s, a), raised once
// a step.  (In places of its own in shared memory, filled two steps ahead, they cost as many
// instructions again: 512 rows of 126464 took 31.0 us, not 26.6.)
// Exponents are powers of two: u = x c log2 e - R is one FMA from the reference R, two
// elements to an instruction.
//
// For the alternatives a thread keeps its largest value with the first piece that holds it.
// These pairs are all different, and each stands for an element, so a value that top_k of
// them reach is a bound: an element below it (smaller, or equal and in a later piece) has
// top_k others before it.  The bound is the top_k-th largest of the pairs of 32 groups of
// threads; only threads whose own pair is at or above it hold such elements, hardly
// more than top_k of them: their pieces alone are read again, and what passes is ranked.
//
// Measured: 512 rows of 126464 bf16, two alternatives: 26.6 us (floor 19.1), of which the stream
// with the launch and the join is 23.4, the alternatives behind it are 1.8, and exponentials
// and sums, which go on beside the loads, the rest; 1500 rows 71 (5.4 TB/s).  333 rows of 32003
// fp32: 13.4 us (6.3), the alternatives again 1.8.  One row, 20 alternatives: 8.0 us, of
// which they are 1.9.
#include <math.h>

#include "layer_ops.cuh"
#include "pairs.cuh"
#include "sm103.cuh"

namespace dllm {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // pieces of a step
constexpr int kMaxCluster = 8;
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
  static __device__ __forceinline__ uint4 none() { return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }
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
      const float2 f = unpack2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ float largest(const uint4& u) {
    const float2 f = unpack2(max_bf16x2(max_bf16x2(u.x, u.y), max_bf16x2(u.z, u.w)));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ void pairs(const uint4& u, float2 (&p)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = unpack2(max_nan_bf16x2(w[i], kLow2));
  }
  static __device__ __forceinline__ uint4 none() { return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
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

// (x - y) c for x <= y, also where x - y is beyond fp32 and the product is not.
__device__ __forceinline__ float scaled_apart(float x, float y, float c) {
  const float d = x - y;
  return d == -INFINITY ? (0.5f * x - 0.5f * y) * c * 2.f : d * c;
}

// Sums of weights 2^(u - r) and of weight x (u - r), u = x c log2 e.  The slow form keeps r in units of x, and works on
// differences of x.
template <bool SLOW>
struct Stat {
  float r, s, a;
  static __device__ __forceinline__ float apart(float x, float y, float c) {
    return SLOW ? fmaxf(scaled_apart(x, y, c), -1000.f) : x - y;
  }
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

// The slow form's sums of all pieces, by one team.
template <typename T, int TEAM>
__device__ __noinline__ Stat<true> slow_sums(const Row<T>& row, float c, int tid) {
  constexpr int N = Piece<T>::N;
  constexpr float kMin = -3.402823466e38f;
  Stat<true> t = {kMin, 0.f, 0.f};
  for (int v = tid; v < row.pieces; v += TEAM) {
    float x[N];
    Piece<T>::get(row.get(v), x);
    Stat<true> p = {kMin, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) p.r = fmaxf(p.r, x[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float u = max_nan(scaled_apart(x[i], p.r, c), -1000.f), e = ex2(u);
      p.s += e;
      p.a = fmaf(e, u, p.a);
    }
    t.join(p, c);
  }
  return t;
}

template <int TEAM>
struct Shared {
  static constexpr int kWarps = TEAM / 32;
  static constexpr int kList = TEAM == 32 ? 256 : 512;  // elements ranked at once
  float ref[kWarps];
  float2 sum[kWarps];
  uint64_t key[TEAM > 32 ? TEAM : 1];  // the threads' pairs
  uint64_t list[kList];
  uint64_t best[kMaxTop];  // the alternatives, largest first
  uint64_t prev, round[kWarps];
  int owners[TEAM], n_owners, n_list;
};
// What the CTAs of a cluster leave with the first one.
struct Parts {
  float stat[kMaxCluster][3];
  uint64_t best[kMaxCluster * kMaxTop];
};

template <int TEAM>
__device__ __forceinline__ void team_sync() {
  if (TEAM == 32)
    __syncwarp();
  else
    __syncthreads();
}

// The sums of a team's threads, in a fixed order, to all of them: the reference first, then all relative to it.
template <int TEAM, bool SLOW>
__device__ __forceinline__ Stat<SLOW> team_join(Stat<SLOW> t, float c, Shared<TEAM>& sh, int tid) {
  constexpr int W = TEAM / 32;
  const int lane = tid & 31, warp = tid >> 5;
  float n = t.r;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
  if (W > 1) {
    if (lane == 0) sh.ref[warp] = n;
    team_sync<TEAM>();
#pragma unroll
    for (int w = 0; w < W; ++w) n = fmaxf(n, sh.ref[w]);
  }
  const float d = Stat<SLOW>::apart(t.r, n, c), f = ex2(d);
  float s = f * t.s, a = f * (t.a + t.s * d);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    a += __shfl_xor_sync(0xffffffffu, a, o);
  }
  if (W > 1) {
    if (lane == 0) sh.sum[warp] = make_float2(s, a);
    team_sync<TEAM>();
    s = a = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      s += sh.sum[w].x;
      a += sh.sum[w].y;
    }
  }
  return {n, s, a};
}

// The want-th largest of a warp's 64-bit values (all different, but for 0: none), or 0 where there are fewer.
__device__ __forceinline__ uint64_t nth_largest(uint64_t g, int want) {
  uint32_t hi = static_cast<uint32_t>(g >> 32), lo = static_cast<uint32_t>(g);
  for (;;) {
    const uint32_t h = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t l = __reduce_max_sync(0xffffffffu, hi == h ? lo : 0u);
    if (h == 0) return 0;
    if (--want == 0) return static_cast<uint64_t>(h) << 32 | l;
    if (hi == h && lo == l) hi = 0;
  }
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <typename T, int TEAM, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, TEAM == 32 ? 3 : 4) token_scores_kernel(const ScoreArgs a, int cluster) {
  constexpr int N = Piece<T>::N, kTeams = kThreads / TEAM;
  using Sh = Shared<TEAM>;
  __shared__ Sh shared[kTeams];
  const int team = static_cast<int>(threadIdx.x) / TEAM, tid = static_cast<int>(threadIdx.x) % TEAM;
  const int lane = tid & 31, warp = tid >> 5;
  Sh& sh = shared[team];
  const int rank = CLUSTER ? static_cast<int>(blockIdx.x) % cluster : 0;
  const int stretch = CLUSTER ? TEAM * cluster : TEAM;
  const float c = fminf(a.scale * kLog2e, 3.402823466e38f);
  if (CLUSTER) cluster_arrive_release();  // this CTA runs: the others may write to it
  griddep_wait();
  griddep_launch_dependents();
  const int j = CLUSTER ? static_cast<int>(blockIdx.x) / cluster : static_cast<int>(blockIdx.x) * kTeams + team;
  if (j >= a.rows) return;  // (a warp's: no barrier of a CTA follows there)
  const Row<T> row(static_cast<const T*>(a.logits) + j * a.stride, a.vocab);
  int tok = -1;  // thread 0: the given token, and its logit on its way
  float tok_x = 0.f;
  if (tid == 0 && rank == 0 && a.tokens != nullptr) {
    tok = __ldg(a.tokens + j);
    if (tok >= 0 && tok < a.vocab) tok_x = Piece<T>::one(row.p + tok);
  }

  // ---- sums, and this thread's largest
  float m = kLow, r = kLow * c, top = -INFINITY;
  int top_v = 0;
  float2 s2 = {0.f, 0.f}, a2 = {0.f, 0.f};
  const int v_first = rank * TEAM + tid;  // this thread's first piece
  const int steps = (row.pieces + kBatch * stretch - 1) / (kBatch * stretch);
  // steps [from, to) have whole pieces only
  const int whole_to = (row.lead + row.n) / N - (kBatch - 1) * stretch - v_first;
  const int to = whole_to > 0 ? (whole_to + kBatch * stretch - 1) / (kBatch * stretch) : 0;
  const int from = row.lead > 0 && v_first == 0 ? 1 : 0;
  const T* next = row.p + static_cast<int64_t>(row.first(v_first));
  auto ask = [&](int i, uint4 (&q)[kBatch]) {
    if (i >= from && i < to) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) q[b] = __ldg(reinterpret_cast<const uint4*>(next + b * stretch * N));
    } else if (i < steps) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int v = v_first + (i * kBatch + b) * stretch;
        q[b] = v >= row.pieces ? Piece<T>::none() : row.whole(v) ? row.load(v) : row.edge(v);
      }
    }
    next += kBatch * stretch * N;
  };
  auto step = [&](int i, const uint4 (&q)[kBatch]) {
    float most = m;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float l = Piece<T>::largest(q[b]);
      most = fmaxf(most, l);
      if (l > top) {
        top = l;
        top_v = i * kBatch + b;
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
      for (int k = 0; k < N / 2; ++k) {
        const float2 u = fma2(p[k], {c, c}, {-r, -r});
        const float2 e = {ex2(u.x), ex2(u.y)};
        s2 = add2(s2, e);
        a2 = fma2(e, u, a2);
      }
    }
  };
  uint4 qa[kBatch], qb[kBatch];
  ask(0, qa);
#pragma unroll 1
  for (int i = 0; i < steps; i += 2) {
    ask(i + 1, qb);
    step(i, qa);
    if (i + 1 < steps) {
      ask(i + 2, qa);
      step(i + 1, qb);
    }
  }
  const uint64_t best = key_of(top, v_first + top_v * stretch);
  Stat<false> t = {r, s2.x + s2.y, a2.x + a2.y};
  t = team_join<TEAM>(t, c, sh, tid);

  // ---- this team's alternatives (the row's largest at least), as keys of element numbers
  const int want = a.top > 0 ? a.top : 1;
  {
    uint64_t g = best;
    if (tid == 0) sh.n_owners = sh.n_list = 0;
    if (tid < kMaxTop) sh.best[tid] = 0;
    if (TEAM > 32) {  // (a group is a lane of all warps: each has something wherever 32 threads do)
      sh.key[tid] = best;
      team_sync<TEAM>();
#pragma unroll
      for (int w = 0; w < TEAM / 32; ++w) g = sh.key[w * 32 + lane] > g ? sh.key[w * 32 + lane] : g;
    }
    const uint64_t bound = nth_largest(g, want);  // (every warp for itself)
    team_sync<TEAM>();
    if (best != 0 && best >= bound) sh.owners[atomicAdd(&sh.n_owners, 1)] = tid;
    team_sync<TEAM>();
    const int no = sh.n_owners, each = (row.pieces + stretch - 1) / stretch;
    for (int i0 = tid; i0 < no * each; i0 += 2 * TEAM) {
      int v[2];
      uint4 u[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = i0 + k * TEAM, q = i / no;
        v[k] = row.pieces;
        if (i < no * each) {
          const int o = sh.owners[i - q * no];
          v[k] = o + rank * TEAM + q * stretch;
          if (v[k] < row.pieces) u[k] = row.get(v[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (v[k] >= row.pieces || key_of(Piece<T>::largest(u[k]), v[k]) < bound) continue;
        float x[N];
        Piece<T>::get(u[k], x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (x[e] > -INFINITY && key_of(x[e], v[k]) >= bound) {
            const int at = atomicAdd(&sh.n_list, 1);
            if (at < Sh::kList) sh.list[at] = key_of(x[e], row.first(v[k]) + e);
          }
        }
      }
    }
    team_sync<TEAM>();
    const int nl = sh.n_list;
    if (nl <= Sh::kList) {
      for (int i = tid; i < nl; i += TEAM) {
        const uint64_t mine = sh.list[i];
        int before = 0;
        for (int o = 0; o < nl; ++o) before += sh.list[o] > mine;
        if (before < want) sh.best[before] = mine;
      }
    } else {  // so many in so few threads' pieces: one after the other
      if (tid == 0) sh.prev = ~0ull;
      team_sync<TEAM>();
      for (int k = 0; k < want; ++k) {
        const uint64_t prev = sh.prev;
        uint64_t most = 0;
        for (int i = tid; i < no * each; i += TEAM) {
          const int v = sh.owners[i % no] + rank * TEAM + i / no * stretch;
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
        team_sync<TEAM>();
        if (tid == 0) {
          for (int w = 1; w < Sh::kWarps; ++w) most = sh.round[w] > most ? sh.round[w] : most;
          sh.prev = sh.best[k] = most;
        }
        team_sync<TEAM>();
      }
    }
    team_sync<TEAM>();
  }

  // ---- the cluster's parts meet in its first CTA
  if constexpr (CLUSTER) {
    __shared__ Parts parts;
    cluster_wait_acquire();
    const uint32_t base = mapa_shared(smem_u32(&parts), 0) - smem_u32(&parts);
    if (tid == 0) {
      st_cluster_f32(base + smem_u32(&parts.stat[rank][0]), t.r);
      st_cluster_f32(base + smem_u32(&parts.stat[rank][1]), t.s);
      st_cluster_f32(base + smem_u32(&parts.stat[rank][2]), t.a);
    }
    if (tid < want) st_cluster_u64(base + smem_u32(&parts.best[rank * want + tid]), sh.best[tid]);
    cluster_arrive_release();
    cluster_wait_acquire();
    if (rank != 0) return;
    t = {parts.stat[0][0], parts.stat[0][1], parts.stat[0][2]};
    for (int i = 1; i < cluster; ++i) t.join({parts.stat[i][0], parts.stat[i][1], parts.stat[i][2]}, c);
    __syncthreads();
    if (tid < kMaxTop) sh.best[tid] = 0;
    __syncthreads();
    if (tid < cluster * want) {
      const uint64_t mine = parts.best[tid];
      int before = 0;
      for (int i = 0; i < cluster * want; ++i) before += parts.best[i] > mine;
      if (mine != 0 && before < want) sh.best[before] = mine;
    }
    __syncthreads();
  }

  // ---- results
  const uint64_t first = sh.best[0];
  const float largest = first != 0 ? value_of(first) : -INFINITY;
  const bool slow = largest != INFINITY && (c < kLeast || c > kMost ||
                                            (first != 0 && (fabsf(largest) > kFar || fabsf(largest) * c > kFar)));
  float ref = t.r, s = t.s, wa = t.a;
  if (slow) {
    const Stat<true> z = team_join<TEAM>(slow_sums<T, TEAM>(row, c, tid), c, sh, tid);
    ref = z.r;
    s = z.s;
    wa = z.a;
  }
  if (warp != 0) return;
  const bool bad = !(s < INFINITY) || largest == INFINITY;  // a NaN or +inf
  const bool empty = !bad && first == 0;
  const float nan = __int_as_float(0x7FFFFFFF), ls = log2f(s);
  // log of the sum relative to the largest; log p of a logit
  const float log_s = ((slow ? 0.f : fmaf(-largest, c, ref)) + ls) * kLn2;
  auto logp = [&](float x) {
    const float d = x - largest;
    return d == -INFINITY && x > -INFINITY ? fmaf(0.5f * x - 0.5f * largest, 2.f * a.scale, -log_s) : fmaf(d, a.scale, -log_s);
  };
  if (tid == 0) {
    if (bad) report_error(a.err, kErrRange);
    if (a.lse != nullptr) a.lse[j] = bad ? nan : empty ? -INFINITY : fmaf(largest, a.scale, log_s);
    if (a.entropy != nullptr) a.entropy[j] = bad ? nan : empty ? 0.f : (ls - wa / s) * kLn2;
    if (a.tokens != nullptr) {
      float lp = 0.f;
      if (tok >= a.vocab) report_error(a.err, kErrBadShape);
      if (bad || tok >= a.vocab)
        lp = nan;
      else if (tok >= 0)
        lp = empty ? -INFINITY : logp(tok_x);
      a.logp[j] = lp;
    }
  }
  if (tid < a.top) {
    const uint64_t key = bad ? 0 : sh.best[tid];
    const int64_t at = static_cast<int64_t>(j) * a.top + tid;
    a.top_ids[at] = key != 0 ? place_of(key) : -1;
    a.top_logp[at] = bad ? nan : key != 0 ? logp(value_of(key)) : -INFINITY;
  }
}

template <typename T, int TEAM, bool CLUSTER>
cudaError_t launch_scores(const ScoreArgs& a, int cluster, cudaStream_t stream) {
  // (64 registers, for four CTAs an SM; of a cluster's, two at most are there, which could have twice as many)
  const auto kernel = token_scores_kernel<T, TEAM, CLUSTER>;
  constexpr int kTeams = kThreads / TEAM;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CLUSTER ? a.rows * cluster : (a.rows + kTeams - 1) / kTeams);
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
  cfg.numAttrs = CLUSTER ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, cluster);
}

template <typename T>
cudaError_t launch_type(const ScoreArgs& a, int num_sms, cudaStream_t stream) {
  // Few rows: a cluster to each, as long as a CTA has a step for each thread (126464 bf16 with 1, 2, 4, 8 CTAs: one row 13.7,
  // 11.0, 8.6, 8.1 us; 32 rows 10.3, 8.5, 6.8, 6.6; 128 rows 13.3, 11.4, 11.0, 15.6; 300 rows 18.2, 18.5, 26.8, 35.0).
  const int pieces = a.vocab / Piece<T>::N;
  int cluster = 1;
  while (cluster < kMaxCluster && static_cast<int64_t>(a.rows) * cluster * 2 <= 2 * num_sms &&
         pieces >= cluster * 2 * kThreads * kBatch)
    cluster *= 2;
  if (cluster > 1) return launch_scores<T, kThreads, true>(a, cluster, stream);
  // Many short rows: a warp to each, which waits for no other (2500 of 4000 bf16: 9.4 us for 28.0; of 16000: 24 for 35).
  // With more alternatives most of a warp's threads hold one, and most of the row is read twice (2500 of 16000, 20
  // alternatives: 51 for 42; of 4000: 20 for 35).
  if (a.rows >= 4 * num_sms && pieces <= (a.top <= 4 ? 2048 : 512)) return launch_scores<T, 32, false>(a, 1, stream);
  return launch_scores<T, kThreads, false>(a, 1, stream);
}

}  // namespace

cudaError_t launch_token_scores(const ScoreArgs& a, int num_sms, cudaStream_t stream) {
  if (a.rows <= 0) return cudaSuccess;
  return a.fp32 ? launch_type<float>(a, num_sms, stream) : launch_type<__nv_bfloat16>(a, num_sms, stream);
}

}  // namespace dllm
