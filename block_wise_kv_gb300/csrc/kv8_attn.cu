// kv8_attn.cu — attention of the block rows over the e4m3 paged cache, on tcgen05.
//
// A unit of work is (sequence, key head, up to NQ of the rows that share it): row r
// is block row r / G under query head h G + r % G, G = query heads to a key head.
// Keys go in tiles of 128 (two pages), and everything is transposed so that the
// 128 keys fill the tensor core's M and the few rows are its N:
//
//   S^T[key][row] = K8 (Q_hi + Q_lo)^T         e4m3 x e4m3, two products into one accumulator
//   P^T[key][row] = 2^(x),  x = f_key g_row S - R_row  (key scale; q scale x softmax scale x log2 e)
//   O^T[col][row] += V8^T (P_hi + P_mid + P_lo)^T  e4m3 x e5m2
//
// The pages are used as they lie: no key or value is ever converted.  What makes that
// exact enough is the other operand.  A row's q is scaled by a power of two of its own so
// that its largest is in (224, 448], and split into two e4m3 parts.  4 + 4 bits hold
// bf16's 8 exactly where the scaled value is 2^-2 or more (at least down to 2^-9.8 of the
// row's largest); smaller ones are off by up to 2^-10, half of e4m3's smallest step (at
// most 2^-17.8 of the row's largest).  With one scale for a whole unit a row lost what it
// was smaller than its neighbours by, and was all zeros at 2^-19 of them; a row's own costs
// a product for each pair of scores (32 ragged sequences 136 us for 131).
// A weight is rounded to fp16 (11 bits) and split into three e5m2 parts, which is
// exact (3 bits each, rounded to nearest) but for an absolute 2^-17, half of the
// smallest e5m2 step, where a row's largest is 2^10 or more: a softmax with one large
// weight and a long flat tail that together weighs as much keeps its tail.  The value
// scale of a key multiplies its weight before the split; the sum l takes the weight
// without it.
//
// The thread that holds a key's scores has its scales as two scalars; a row's g and
// reference R are the same for all 128 keys.  R is set from a unit's first tile (so
// that the largest weight x value scale is 2^10) and raised only when one passes 2^15:
// a vote per tile, and otherwise no reduction over keys at all until the unit's end,
// where the 128 partial sums of each row are added.
//
// Roles of a CTA's warps: groups of four softmax warps (TMEM lane = key, then = column
// of O^T; 16 rows to a group, 32 in units of 64), one TMA producer, one MMA issuer.  K
// and V tiles share one ring of 16 KB slots (8 KB for d = 64).  The tensor core has the
// next tile's S done, from the moment the scores are in registers, while the softmax
// works.  Two or three CTAs an SM cover each other's serial parts.
//
// Split: the tiles of all units form one line, cut into as many equal pieces as CTAs
// (or fewer, where there are few tiles): a ragged batch or one long sequence loads all
// SMs alike.  Each unit stands there with two or three more than it has: what q, the first
// reference and the output cost.  (Without them the CTAs that got the many short units of
// a ragged batch took 1.6 times the mean.)  A unit cut by a border leaves its pieces'
// (O, R, l) in the workspace, and a second, small kernel joins them in the order of the
// keys, a warp for each row (not launched, and no unit cut, where no sequence has more
// than kWholeTiles tiles): with the ring full, every dependent trip to memory (fence,
// counter, reads) costs the attention's warps several microseconds, which a join inside
// the kernel had to wait for.
//
// Bound and measured (d = 128): single tokens and long contexts by HBM (64 sequences of up
// to 16384 keys, 8 key heads: 151 us, 6.6 TB/s; two of 131072: 83 us, 6.0 TB/s with the
// join).  Wider units by the chain of a tile (scores, vote, weights, products), 1.9 us a
// tile and CTA for 64 rows, 1.4 for 32, with 16 softmax warps an SM (what the registers
// hold) and the issue slots half busy: 32 ragged sequences of up to 4608 keys, blocks of
// 16 to 64: 136 us, 4.3 TB/s; eight sequences with 128 rows to a key head: 43 us.  16
// sequences of 1536 with blocks of 32: 44 us, 4.7 TB/s.  One sequence of 768: 12 us, of
// which the two launches take 3.4, the line 1.1, the join 3.7.  Half the columns are half
// the bytes of a tile and the same chain: the 16 sequences as 64 heads of 64 take 70 us.
// All of these are with scores whose spread is about 1.3 (in natural units), where R is
// hardly ever raised.  With queries 2, 4 and 8 times as large the 16 sequences take 48, 54
// and 56 us, the ragged ones 168, 204 and 218.
#include <algorithm>

#include "attn_common.cuh"
#include "kv8.cuh"

namespace dllm {
namespace {

constexpr int kTile = 128;  // keys per tile: two pages
constexpr int kScaleSlots = 8;       // tiles whose scales are in shared memory
constexpr int kMaxCtas = 1024;       // of a launch (records of the workspace)
constexpr size_t kRecordBytes = kMaxCtas * sizeof(int2);
// Sequences of up to this many tiles are not cut: three more tiles in a row take about what the second launch does
// (320 tokens of 4 heads: 9.4 us cut and joined, 8.5 whole, and 2 us less on the host).
constexpr int kWholeTiles = 4;
// Up to this many sequences are summed up by the producer warp alone, four a lane; beyond, by as many threads through
// shared memory, behind a barrier of the CTA (with that way for 16 sequences: 45.5 us for 44.2, one sequence 12.7 for 11.9).
constexpr int kScan = 128;
constexpr int kParts = 16;           // parts of units in shared memory: the producer is fewer than 8 tiles ahead
constexpr float kTop = 10.f;    // log2 of a row's largest weight x value scale when R is set
constexpr float kLimitLog2 = 15.f;
constexpr float kLimit = 32768.f;  // what a weight x value scale may reach before R is raised

// What a unit's beginning and end cost, in tiles (see the split above): 32 ragged sequences in units of 64 take 145 us
// with 2, 136 with 3, 138 with 4; 16 of 1536 in units of 32 44.9 with 1, 44.3 with 2, 44.7 with 3; 64 of single tokens in
// units of 16 151 with 1 or 2, 153 with 3.
__host__ __device__ constexpr int unit_tiles(int nq) { return nq == 64 ? 3 : 2; }

// CTAs an SM (of a unit's width): with 16 rows, memory's latency is what more of them cover, 96 registers a thread nearly
// do (40 bytes go to the stack and back), and three slots of the ring hold a tile and the next key tile (64 sequences of up
// to 16384 keys: 157.7 us with two, 151.4 with three, 150.5 with four, whose rings have two slots; two of 131072 keys: 84.9,
// 82.8, 84.5).  Wider units' softmax needs the registers: 32 rows took 45.0 us with two CTAs of 16 rows a thread, 49.0 with
// three of 32 rows a thread.
constexpr int ctas_per_sm(int nq) { return nq == 16 ? 3 : 2; }

// NQ rows to a unit, handled by NQ / kCols groups of four softmax warps (a thread: one key, kCols rows).
template <int D, int NQ>
struct Cfg {
  static constexpr int kCols = NQ == 64 ? 32 : 16;
  static constexpr int kCtas = ctas_per_sm(NQ);
  static constexpr int kGroups = NQ / kCols;
  static constexpr int kSoft = 128 * kGroups;  // softmax threads
  static constexpr uint32_t kTmemCols = 4 * NQ;  // S^T, O^T of the three parts
  static constexpr int kProducerWarp = 4 * kGroups, kMmaWarp = kProducerWarp + 1;
  static constexpr int kThreads = kSoft + 64;
  static constexpr int kSlotBytes = kTile * D;
  static constexpr int kQBytes = NQ * D * 2;                  // hi, lo
  // P^T's rows of 64 or 128 bytes: up to NQ = 32 the three parts of a weight side by side, else three planes.
  static constexpr bool kPlanes = NQ == 64;
  static constexpr int kPRow = NQ == 32 ? 128 : 64;
  static constexpr int kPBytes = kTile * kPRow * (kPlanes ? 3 : 1);
  static constexpr int kStatic = NQ == 64 ? 6400 : NQ == 32 ? 4608 : 3584;  // static shared memory, at most
  static constexpr int kBudget = 227 * 1024 / kCtas - 2048 - kStatic;  // 1 KB to align, 1 KB of the system's a CTA
  static constexpr int kSlots0 = (kBudget - kQBytes - kPBytes) / kSlotBytes;
  static constexpr int kSlots = kSlots0 > 10 ? 10 : kSlots0;
  static constexpr int kDynSmem = kSlots * kSlotBytes + kQBytes + kPBytes + 1024;
  static_assert(kSlots >= 2, "a tile's V needs a slot beside the next tile's K");
  static_assert(kSlots / 2 + 2 < kScaleSlots, "scales stay until the softmax has read them");
  static constexpr size_t kPartFloats = static_cast<size_t>(NQ) * (D + 4);  // O, R, l, rows
};

// ------------------------------------------------------------ descriptors
// Tiles of 64- or 128-byte rows with the swizzle of that width: 8-row atoms one after the other.
// `block`: bytes from one row's worth of the contiguous dimension to the next, where an operand has more than one.
template <int ROW>
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t block = 0) {
  static_assert(ROW == 64 || ROW == 128, "swizzled rows");
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(block >> 4) << 16;    // leading byte offset
  d |= static_cast<uint64_t>(ROW * 8 >> 4) << 32;  // stride byte offset: one 8-row atom
  d |= static_cast<uint64_t>(1) << 46;             // descriptor version for tcgen05
  d |= static_cast<uint64_t>(ROW == 128 ? 2 : 4) << 61;
  return d;
  // (V of d = 64 is taken as M = 128 with a leading offset of 0: lanes 64-127 of O^T repeat lanes 0-63 and are not read)
}
// kind::f8f6f4, fp32 accumulator: A e4m3, B e4m3 or e5m2; either operand K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_f8(int m, int n, bool b_e5m2, bool mn) {
  return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((mn ? 1u : 0u) << 15) | ((mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
// Byte offset of 16-byte chunk c of row r in a tile of swizzled ROW-byte rows.
template <int ROW>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return ROW == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Barrier `id` of N threads that ORs a predicate over them.
template <int N>
__device__ __forceinline__ bool barrier_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %3, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "n"(N), "r"(id)
      : "memory");
  return r != 0;
}

// Pairs of fp32 (one instruction for both).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two fp16 to two e4m3 codes (nearest even) and back.
__device__ __forceinline__ uint32_t e4m3x2_of(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// Reduce N values over the warp's lanes: every lane i mod N gets the result of v[i] (v is destroyed).
template <int N, class Op>
__device__ __forceinline__ float reduce_transposed(float (&v)[N], int lane, Op op) {
#pragma unroll
  for (int w = N / 2; w > 0; w >>= 1) {
    const bool up = (lane & w) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float keep = up ? v[i + w] : v[i], give = up ? v[i] : v[i + w];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, w));
    }
  }
  if (N == 16) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
  return v[0];
}
// A thread's N columns of its TMEM lane.
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[16]) { tmem_ld_32x32b_x16(taddr, v); }
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[32]) { tmem_ld_32x32b_x32(taddr, v); }
__device__ __forceinline__ void tmem_store(uint32_t taddr, const float (&v)[16]) { tmem_st_32x32b_x16(taddr, v); }

// The sum of sixteen columns of three blocks `step` columns apart (three loads under way, one wait).
__device__ __forceinline__ void tmem_load3(uint32_t taddr, uint32_t step, float (&v)[16]) {
  uint32_t r[3][16];
#pragma unroll
  for (int z = 0; z < 3; ++z)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[z][0]), "=r"(r[z][1]), "=r"(r[z][2]), "=r"(r[z][3]), "=r"(r[z][4]), "=r"(r[z][5]), "=r"(r[z][6]),
          "=r"(r[z][7]), "=r"(r[z][8]), "=r"(r[z][9]), "=r"(r[z][10]), "=r"(r[z][11]), "=r"(r[z][12]), "=r"(r[z][13]),
          "=r"(r[z][14]), "=r"(r[z][15])
        : "r"(taddr + z * step)
        : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int c = 0; c < 16; ++c) v[c] = (__uint_as_float(r[0][c]) + __uint_as_float(r[1][c])) + __uint_as_float(r[2][c]);
}

// One lane of the warp, which is converged.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Wait for the phase with the given parity, at most 2^18 tries of up to 20 us each (seconds), in few instructions: the
// kernel's roles share the instruction cache.  False where it gave up.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < (1 << 18); ++i)
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
  return false;
}

// ------------------------------------------------------------ work
// The workspace: for each CTA the record (pieces, rows) of the unit that begins in it and goes on in the next, (0, -) if
// none does; then two parts for each CTA: of the unit that began before it, and of the one that goes on after it.

struct Seq {
  int n, s, rows, cub, cus;
  int npages, tiles, nqt;  // tiles = 0: nothing to do
  int bad;                 // (all of them ints: a Seq goes from lane to lane)
};
template <int NQ>
__device__ __forceinline__ Seq load_seq(const Kv8AttnArgs& a, int b) {
  const BatchArgs& bt = a.bt;
  Seq q;
  q.n = __ldg(bt.seq_len + b);
  q.s = __ldg(bt.block_start + b);
  q.rows = __ldg(bt.block_len + b);
  q.cub = __ldg(bt.cu_block + b);
  q.cus = __ldg(bt.cu_seq + b);
  const int next = __ldg(bt.cu_block + b + 1);  // the block's rows are its own: a plan may have counted none of them
  q.tiles = q.nqt = q.npages = 0;
  q.bad = 0;
  if (q.rows == 0 || q.n == 0) return q;
  if (q.n < 0 || q.n > bt.max_seq_len || q.rows < 0 || q.rows > bt.max_block_len || q.s < 0 || q.rows > q.n - q.s ||
      q.cub < 0 || next < q.cub || q.rows > min(next, bt.total_block_rows) - q.cub || (q.n + kPage - 1) / kPage > bt.max_pages ||
      (a.full_rows && (q.cus < 0 || q.n > bt.total_seq_rows - q.cus))) {
    q.bad = 1;
    return q;
  }
  q.npages = (q.n + kPage - 1) / kPage;
  q.tiles = (q.n + kTile - 1) / kTile;
  q.nqt = (q.rows * (a.n_heads / a.kv.n_kv_heads) + NQ - 1) / NQ;
  return q;
}
template <int NQ>
__device__ __forceinline__ long long seq_work(const Kv8AttnArgs& a, const Seq& q) {
  return q.tiles == 0 ? 0 : static_cast<long long>(a.kv.n_kv_heads) * q.nqt * (q.tiles + unit_tiles(NQ));
}

// a / b for a >= 0, b > 0 (almost always of 31 bits).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 31) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// A part of a unit as the producer hands it to the other roles.
struct Part {
  int n;             // keys of the sequence
  int t0, t1;        // the part's tiles; t1 = 0: there is no further part
  int tiles;         // of the unit
  int h, r0, cols;   // key head; the unit's first row and its rows
  int cub, s, cus;   // the sequence's places
  int c_last;        // the CTA that has the unit's last tile
};

// A CTA's piece [lo, hi) of the line of tiles, walked unit by unit (by the producer).
template <int NQ>
struct Walk {
  const Kv8AttnArgs& a;
  long long base, pos, hi;  // where sequence b begins on the line; the next tile; the end
  int b;
  Seq q;
  bool whole;      // units are not cut: the piece has those that begin in it
  // the current part of a unit: tiles [t0, t1) of (b, h, qt), whose first tile lies at u0 on the line
  int h, qt, t0, t1;
  long long u0;
  __device__ Walk(const Kv8AttnArgs& args, int b0, const Seq& q0, long long base0, long long lo, long long hi0)
      : a(args), base(base0), pos(lo), hi(hi0), b(b0), q(q0), whole(args.whole_units != 0) {}
  __device__ bool next() {
    int span, x;
    for (;;) {
      if (pos >= hi) return false;
      long long w = seq_work<NQ>(a, q);
      while (pos >= base + w) {
        base += w;
        q = load_seq<NQ>(a, ++b);
        w = seq_work<NQ>(a, q);
      }
      span = q.tiles + unit_tiles(NQ);
      x = static_cast<int>(quotient(pos - base, span));  // unit of the sequence
      const long long begins = base + static_cast<long long>(x) * span;
      if (!whole || pos == begins) break;
      pos = begins + span;  // it began in the piece before
    }
    h = x / q.nqt;
    qt = x % q.nqt;
    u0 = base + static_cast<long long>(x) * span + unit_tiles(NQ);
    t0 = static_cast<int>(max(pos - u0, 0ll));
    t1 = whole ? q.tiles : static_cast<int>(min(static_cast<long long>(q.tiles), hi - u0));
    if (t1 <= 0) return false;  // the piece ends before the unit's first tile
    pos = u0 + t1;
    return true;
  }
};

// ------------------------------------------------------------ the kernel
template <int D, int NQ>
__global__ void __launch_bounds__(Cfg<D, NQ>::kThreads, Cfg<D, NQ>::kCtas)
    kv8_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const Kv8AttnArgs a) {
  using C = Cfg<D, NQ>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* const smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t ring = smem_u32(smem), p_base = ring + C::kSlots * C::kSlotBytes, q_base = p_base + C::kPBytes;
  __shared__ uint64_t full_bar[C::kSlots], empty_bar[C::kSlots], s_full, s_free, p_ready, pv_done, q_ready;
  __shared__ uint64_t scale_bar[kScaleSlots], drain_bar;
  __shared__ uint32_t tmem_sh;
  __shared__ __align__(16) float scales[kScaleSlots][2][8];  // K, V: two pages of four groups
  __shared__ Part part_sh[kParts];
  __shared__ uint64_t part_bar[kParts];
  // of each row: -R; what the sums so far are multiplied by where R is raised; the sum l and 1 / l
  // (two of what the end of a unit still reads when the next has begun)
  __shared__ __align__(16) float nref_sh[2][NQ], alpha_sh[NQ], l_sh[NQ], inv_sh[NQ];
  __shared__ __align__(16) float fq_sh[NQ];  // a row's q scale x softmax scale x log2 e
  __shared__ float red_sh[4][NQ];
  __shared__ long long row_sh[2][NQ];  // row and head of the output, as one index
  __shared__ long long seg_sh[kScan + 1];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const BatchArgs& bt = a.bt;
  if (tid == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&s_free, 4 * C::kGroups);
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(&scale_bar[i], 1);
    for (int i = 0; i < kParts; ++i) mbar_init(&part_bar[i], 1);
    mbar_init(&drain_bar, 1);
    mbar_init(&p_ready, C::kSoft);
    mbar_init(&pv_done, 1);
    mbar_init(&q_ready, C::kSoft);
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == C::kMmaWarp) tmem_alloc(&tmem_sh, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  // what lies above needs nothing from the kernel before this one; the roles go apart from here, but for large batches
  griddep_wait();
  griddep_launch_dependents();

  // ---- the line of tiles: its length T, and the sequence in which this CTA's piece begins (for the producer warp)
  const int cta = blockIdx.x;
  long long T = 0, len = 1, lo = 0, start_base = 0;
  int start_b = 0;
  Seq start_q = {};
  auto cut = [&]() {  // into pieces of len
    len = quotient(T + gridDim.x - 1, gridDim.x);
    lo = min(cta * len, T);
  };
  if (bt.batch <= kScan) {
    if (warp == C::kProducerWarp) {  // up to four sequences a lane
      constexpr int kEach = kScan / 32;
      const int per = (bt.batch + 31) / 32;
      Seq q[kEach];
      long long w[kEach], sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        w[i] = 0;
        const int b = lane * per + i;
        q[i] = Seq{};
        if (i >= per || b >= bt.batch) continue;
        q[i] = load_seq<NQ>(a, b);
        if (q[i].bad && cta == 0) report_error(bt.err, kErrBadShape);
        w[i] = seq_work<NQ>(a, q[i]);
        sum += w[i];
      }
      long long incl = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      T = __shfl_sync(0xffffffffu, incl, 31);
      cut();
      long long at = incl - sum;
      int b = lane * per;
      const unsigned mine = __ballot_sync(0xffffffffu, at <= lo && lo < incl);
      Seq here = q[0];
      bool passing = true;  // the lane's sequences that end at or before lo
#pragma unroll
      for (int i = 0; i < kEach - 1; ++i) {
        passing = passing && lo >= at + w[i];
        if (passing) {
          at += w[i];
          ++b;
          here = q[i + 1];
        }
      }
      const int src = mine != 0 ? __ffs(mine) - 1 : 0;
      start_b = __shfl_sync(0xffffffffu, b, src);
      start_base = __shfl_sync(0xffffffffu, at, src);
      int* const to = reinterpret_cast<int*>(&start_q);
      const int* const from = reinterpret_cast<const int*>(&here);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(Seq) / sizeof(int)); ++i) to[i] = __shfl_sync(0xffffffffu, from[i], src);
    }
  } else {
    const int per = (bt.batch + kScan - 1) / kScan;
    if (tid < kScan) {
      long long w = 0;
      for (int b = tid * per; b < min(bt.batch, (tid + 1) * per); ++b) {
        const Seq q = load_seq<NQ>(a, b);
        if (q.bad && cta == 0) report_error(bt.err, kErrBadShape);
        w += seq_work<NQ>(a, q);
      }
      seg_sh[tid] = w;
    }
    __syncthreads();
    if (warp == C::kProducerWarp) {
      constexpr int kEach = kScan / 32;
      long long w[kEach], sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        w[i] = seg_sh[lane * kEach + i];
        sum += w[i];
      }
      long long incl = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      T = __shfl_sync(0xffffffffu, incl, 31);
      cut();
      long long at = incl - sum;
      const unsigned mine = __ballot_sync(0xffffffffu, at <= lo && lo < incl);
      int b = lane * kEach * per;
      if (at <= lo && lo < incl) {
#pragma unroll 1
        for (;; ++b) {
          const long long next = at + seq_work<NQ>(a, load_seq<NQ>(a, b));
          if (lo < next) break;
          at = next;
        }
      }
      const int src = mine != 0 ? __ffs(mine) - 1 : 0;
      start_b = __shfl_sync(0xffffffffu, b, src);
      start_base = __shfl_sync(0xffffffffu, at, src);
      if (lo < T) start_q = load_seq<NQ>(a, start_b);
    }
  }
  // the ring's order: K of the next tile before V of this one, which is needed later (the last tile's V leaves the place
  // of the K that does not follow empty)
  auto k_index = [](int n) { return n == 0 ? 0 : 2 * n - 1; };
  auto v_index = [](int n) { return 2 * n + 2; };
  const int G = a.n_heads / a.kv.n_kv_heads;

  if (warp == C::kProducerWarp) {
    // ------------------------------------------------------------ TMA producer
    // The copies of a tile are issued by lanes of one instruction each (K or V: a page a lane; the four pieces of scales):
    // a single thread that issued them one after the other was the slowest part of the CTA.
    const long long hi = min(lo + len, T);
    Walk<NQ> walk(a, start_b, start_q, start_base, lo, hi);
    int slot = 0, phase = 0, issued = 0, nt = 0, n_parts = 0;
    bool ok = true;
    auto hand_over = [&](bool any) {  // the walk's part, or that there is no more
      if (lane == 0) {
        Part& p = part_sh[n_parts % kParts];
        p.t1 = 0;
        if (any) {
          const Seq& q = walk.q;
          const int r0 = walk.qt * NQ;
          p = Part{q.n, walk.t0, walk.t1, q.tiles, walk.h, r0, min(NQ, q.rows * G - r0), q.cub, q.s, q.cus,
                   static_cast<int>(quotient(walk.u0 + q.tiles - 1, len))};
        }
        mbar_arrive(&part_bar[n_parts % kParts]);
      }
      ++n_parts;
    };
    uint64_t once, again;  // keys that no other unit reads, and others
    once = l2_evict_first_policy();
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
    auto page_ids = [&](const int32_t* row, int first, int npages) {  // of 16 tiles, one a lane (checked where used)
      const int p = first + lane;
      return p < npages ? __ldg(row + p) : 0;
    };
    const int page = lane & 1;
    auto next_slot = [&]() {
      ++issued;
      if (++slot == C::kSlots) {
        slot = 0;
        phase ^= 1;
      }
    };
    auto load_codes = [&](const CUtensorMap* map, int pages, int y, uint64_t policy) {
      if (issued >= C::kSlots) ok = wait_phase(&empty_bar[slot], phase ^ 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) report_error(bt.err, kErrTimeout);
        return;
      }
      if (lane == 0) mbar_arrive_expect_tx(&full_bar[slot], pages * (kPage * D));
      __syncwarp();
      if (lane < pages) tma_load_2d_hint(smem + slot * C::kSlotBytes + page * (kPage * D), map, &full_bar[slot], 0, y, policy);
      next_slot();
    };
    int y_last = 0, pages_last = 0;  // the last tile, whose V is still to be asked for
    uint64_t policy_last = again;
    bool have = walk.next();
    int ids_next = have ? page_ids(bt.block_table + static_cast<size_t>(walk.b) * bt.max_pages, 2 * walk.t0, walk.q.npages) : 0;
    hand_over(have);
    while (have && ok) {
      // this part's values: the walk goes on to the next before its end, whose page ids and rows of q are asked for ahead
      const int32_t* const row = bt.block_table + static_cast<size_t>(walk.b) * bt.max_pages;
      const int t0 = walk.t0, t1 = walk.t1, h = walk.h, npages = walk.q.npages;
      const uint64_t policy = walk.q.nqt > 1 ? again : once;
      int ids = ids_next, first = 2 * t0;
      for (int t = t0; t < t1 && ok; ++t) {
        if (2 * t - first >= 32) {
          first = 2 * t;
          ids = page_ids(row, first, npages);
        }
        const int pages = min(2, npages - 2 * t);
        int id = __shfl_sync(0xffffffffu, ids, 2 * t + page - first);
        if (id < 0 || id >= bt.num_pages) {
          if (lane < 2) report_error(bt.err, kErrBadPage);
          id = 0;
        }
        const int unit = id * a.kv.n_kv_heads + h;  // 64 units of rows fit 31 bits
        load_codes(&tm_k, pages, unit * kPage, policy);
        if (!ok) break;
        const int z = nt % kScaleSlots;
        if (lane == 0) mbar_arrive_expect_tx(&scale_bar[z], pages * 32);
        __syncwarp();
        if (lane < 4 && page < pages)  // lanes 0, 1: K's, 2, 3: V's
          bulk_load(&scales[z][lane >> 1][4 * page], (lane < 2 ? a.kv.k_scale : a.kv.v_scale) + static_cast<size_t>(unit) * kKv8Groups,
                    16, &scale_bar[z]);
        if (nt > 0) load_codes(&tm_v, pages_last, y_last, policy_last);
        y_last = unit * kPage;
        pages_last = pages;
        policy_last = policy;
        ++nt;
        if (t == t0) {  // the next part, while this one's first tile is on its way
          have = walk.next();
          hand_over(have);
          if (have) {
            ids_next = page_ids(bt.block_table + static_cast<size_t>(walk.b) * bt.max_pages, 2 * walk.t0, walk.q.npages);
            for (int c = lane; c < NQ; c += 32) {
              const int r = walk.qt * NQ + c;
              if (r >= walk.q.rows * G) break;
              const char* src = reinterpret_cast<const char*>(static_cast<const __nv_bfloat16*>(a.q) + (walk.q.cub + r / G) * a.q_row +
                                                              static_cast<size_t>(walk.h * G + r % G) * D);
              for (int z = 0; z < D * 2; z += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + z));
            }
          }
        }
      }
    }
    if (ok && nt > 0) {
      next_slot();
      load_codes(&tm_v, pages_last, y_last, policy_last);
    }
    if (lane == 0) {  // every copy has landed and every slot's last release has arrived before the CTA ends
      for (int i = max(0, nt - kScaleSlots); i < nt; ++i)
        if (!wait_phase(&scale_bar[i % kScaleSlots], (i / kScaleSlots) & 1)) report_error(bt.err, kErrTimeout);
      const int none = ok ? 2 * nt - 1 : -1;
      for (int i = max(0, issued - C::kSlots); i < issued; ++i)
        if (i != none && !wait_phase(&full_bar[i % C::kSlots], (i / C::kSlots) & 1)) report_error(bt.err, kErrTimeout);
      for (int i = max(0, issued - C::kSlots); ok && i < issued; ++i)
        if (i != none && !wait_phase(&empty_bar[i % C::kSlots], (i / C::kSlots) & 1)) report_error(bt.err, kErrTimeout);
    }
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // All of the warp goes through the loop, and its conditions are the same for every lane by votes: descriptors and
    // counters can stay in the warp's uniform registers, which is where a product takes them from.  (One lane alone: 0.4 us
    // more for 16 sequences of 1536 keys and for 128 rows to a key head.)
    constexpr uint32_t kIdescS = idesc_f8(kTile, NQ, false, false);
    constexpr uint32_t kIdescO = idesc_f8(kTile, 3 * NQ, true, true);
    const uint32_t tm_o = tmem + NQ;
    const uint64_t q_desc = desc_rows<D>(q_base), p_desc = desc_rows<C::kPRow>(p_base, C::kPlanes ? kTile * C::kPRow : 0);
    int nt = 0, unit = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      if (ok) ok = __all_sync(0xffffffffu, wait_phase(bar, parity & 1));
      return ok;
    };
    auto issue_pv = [&](int n, bool fresh) {  // tile number n of this CTA; the first of its part
      const int i = v_index(n), s = i % C::kSlots;
      if (!wait(&p_ready, n) || !wait(&full_bar[s], i / C::kSlots)) return;
      tc_fence_after();
      const uint64_t v = desc_rows<D>(ring + s * C::kSlotBytes);  // (a step of n bytes adds n / 16 to the address field)
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 32; ++k) umma_e4m3(tm_o, v + k * 2 * D, p_desc + k * 2 * C::kPRow, kIdescO, !fresh || k > 0);
        umma_commit(&empty_bar[s]);
        umma_commit(&pv_done);
      }
      __syncwarp();
    };
    for (;; ++unit) {
      if (!wait(&part_bar[unit % kParts], unit / kParts)) break;
      const Part& part = part_sh[unit % kParts];
      const int tiles = __reduce_max_sync(0xffffffffu, part.t1 == 0 ? 0 : part.t1 - part.t0);
      if (tiles == 0 || !wait(&q_ready, unit)) break;
      for (int t = 0; t < tiles && ok; ++t, ++nt) {
        const int i = k_index(nt), s = i % C::kSlots;
        if (!wait(&full_bar[s], i / C::kSlots)) break;
        if (nt > 0 && !wait(&s_free, nt - 1)) break;
        tc_fence_after();
        const uint64_t k8 = desc_rows<D>(ring + s * C::kSlotBytes);
        if (elect_one()) {
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              umma_e4m3(tmem, k8 + k * 2, q_desc + (part * NQ * D + k * 32) / 16, kIdescS, part > 0 || k > 0);
          umma_commit(&empty_bar[s]);
          umma_commit(&s_full);
        }
        __syncwarp();
        if (t > 0) issue_pv(nt - 1, t == 1);
      }
      if (ok) issue_pv(nt - 1, tiles == 1);
    }
    // the softmax warps wait for the last S and P V, the producer for the releases; where a wait gave up, the
    // products that were issued end before the CTA does
    if (!ok) {
      if (lane == 0) report_error(bt.err, kErrTimeout);
      if (elect_one()) umma_commit(&drain_bar);
      __syncwarp();
      if (!wait_phase(&drain_bar, 0) && lane == 0) report_error(bt.err, kErrTimeout);
    }
  } else {
    // ------------------------------------------------------------ softmax
    constexpr int kCols = C::kCols;
    const int key = tid & 127, grp = tid >> 7, col0 = grp * kCols;  // this thread's key of a tile (column of O^T), and rows
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + lane_base + col0, tm_o = tm_s + NQ;
    // barrier 1 is all softmax warps', 2 + grp a group's: R is a row's own, so groups go through a unit's tiles apart
    auto soft_sync = []() { named_barrier(1, C::kSoft); };
    auto group_sync = [grp]() { named_barrier(2 + grp, 128); };
    int nt = 0;
    bool dead = false;
    auto wait = [&](uint64_t* bar, int parity) {  // a thread that gave up waits for nothing more, but meets every barrier
      if (!dead && !wait_phase(bar, parity & 1)) {
        report_error(bt.err, kErrTimeout);
        dead = true;
      }
    };
    int2 record = make_int2(0, 0);

    // The rows of q of part u: asked for while the last tile of the part before is still to be done (in narrow units, where
    // there are registers for it).
    constexpr int kPer = C::kSoft / NQ, kVec = D / 8 / kPer;  // threads and 16-byte pieces a row
    constexpr bool kAhead = NQ <= 32;
    const int q_row = tid / kPer, q_piece = (tid % kPer) * kVec;
    uint4 qv[kVec];
    auto ask_q = [&](int u) {
      wait(&part_bar[u % kParts], u / kParts);
      const Part& part = part_sh[u % kParts];
      const bool on = !dead && part.t1 > 0 && q_row < part.cols;
      const int r = part.r0 + q_row, i = r / G;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (part.cub + i) * a.q_row +
                                 static_cast<size_t>(part.h * G + r - i * G) * D;
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        qv[k] = on ? __ldg(reinterpret_cast<const uint4*>(src) + q_piece + k) : make_uint4(0, 0, 0, 0);
    };

    // One turn: the next part's q, then the end of the part before it, then the next part's tiles.  So the tensor core
    // has the next scores to work on while the end goes on.
    uint64_t l[kCols / 2];  // sums of pairs of rows over this thread's keys
    for (int u = 0;; ++u) {
      const Part& part = part_sh[u % kParts];
      const int par = u & 1;
      if (!kAhead || u == 0) ask_q(u);
      const bool have = !barrier_any<C::kSoft>(1, dead || part.t1 == 0);  // (the same for all, whoever gave up)
      if (have) {
        // the row's largest: its kPer lanes are neighbours
        auto row_max = [](uint32_t v) {
#pragma unroll
          for (int o = 1; o < kPer; o <<= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
          return v;
        };
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          m = max_u16x2(m, max_u16x2(max_u16x2(qv[i].x & 0x7fff7fffu, qv[i].y & 0x7fff7fffu),
                                     max_u16x2(qv[i].z & 0x7fff7fffu, qv[i].w & 0x7fff7fffu)));
        m = row_max(max(m & 0xffffu, m >> 16));
        if (__any_sync(0xffffffffu, m >= 0x7f80u)) {  // values that are not finite take no part, and make their row not a number
          m = 0;
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            uint32_t* const w = reinterpret_cast<uint32_t*>(&qv[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
              m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
              w[k] |= (lo < 0x7f80u ? 0u : 0x7fu) | (hi < 0x7f80u ? 0u : 0x7f0000u);
            }
          }
          m = row_max(m);
        }
        if (tid < NQ) {
          const int r = part.r0 + tid, i = r / G;
          row_sh[par][tid] = static_cast<long long>(a.full_rows ? part.cus + part.s + i : part.cub + i) * a.n_heads + part.h * G +
                             (r - i * G);
          nref_sh[par][tid] = 0.f;
        }
        // q in two e4m3 parts: 2^e with the row's largest x 2^-e in (224, 448]; 448 = 1.75 2^8
        int e = static_cast<int>(m >> 7) - 127 - ((m & 127u) <= 96u ? 8 : 7);
        e = max(e, -118);
        const float down = __int_as_float((127 - e) << 23);
        if (tid % kPer == 0) fq_sh[q_row] = a.scale_log2 * __int_as_float((127 + e) << 23);
        const uint64_t down2 = pack2(down, down);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
          uint32_t hi2[2], lo2[2];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = unpack2(mul2(pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u)), down2));
            // 8 bits fit fp16's 11, down to 2^-24 of a unit whose last e4m3 step is 2^-9
            const uint32_t h = pack_f16x2(v.x, v.y);
            const uint32_t hc = e4m3x2_of(h), back = f16x2_of(hc);
            const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&back));
            const uint32_t lc = e4m3x2_of(*reinterpret_cast<const uint32_t*>(&rest));
            if (k & 1) {
              hi2[k >> 1] |= hc << 16;
              lo2[k >> 1] |= lc << 16;
            } else {
              hi2[k >> 1] = hc;
              lo2[k >> 1] = lc;
            }
          }
          const int byte = (q_piece + i) * 8;  // eight codes of row q_row
          const uint32_t at = q_base + swz<D>(q_row, byte >> 4) + (byte & 8);
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(hi2[0]), "r"(hi2[1]) : "memory");
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + NQ * D), "r"(lo2[0]), "r"(lo2[1]) : "memory");
        }
        fence_async_smem();
        mbar_arrive(&q_ready);
        if (u == 0) soft_sync();  // the rows' values are there (later ones behind the barriers of the end below)
      }
      if (u > 0) {
        // ---- the end of the part before: l over all keys, then O / l, or (O, R, l) to the workspace
        const Part& done = part_sh[(u - 1) % kParts];
        const int cols = done.cols, was = par ^ 1;
        {
          float v[kCols];
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) {
            const float2 p = unpack2(l[c]);
            v[2 * c] = p.x;
            v[2 * c + 1] = p.y;
          }
          const float sum = reduce_transposed(v, lane, [](float p, float r) { return p + r; });
          if (lane < kCols) red_sh[warp & 3][col0 + lane] = sum;
        }
        soft_sync();
        if (tid < NQ) {
          const float sum = (red_sh[0][tid] + red_sh[1][tid]) + (red_sh[2][tid] + red_sh[3][tid]);
          l_sh[tid] = sum;
          inv_sh[tid] = 1.f / sum;
        }
        wait(&pv_done, nt - 1);
        soft_sync();
        tc_fence_after();
        const bool began = done.t0 == 0, whole = began && done.t1 == done.tiles;
        float* const mine = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + kRecordBytes) +
                            (static_cast<size_t>(cta) * 2 + (began ? 1 : 0)) * C::kPartFloats;
#pragma unroll 1
        for (int c0 = col0; c0 < col0 + kCols; c0 += 16) {
          float o[16];  // column `key` of sixteen rows
          tmem_load3(tm_o + c0 - col0, NQ, o);
          if (key >= D) continue;
          if (whole) {
            __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.o) + key;
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (c0 + c < cols) out[row_sh[was][c0 + c] * D] = __float2bfloat16(o[c] * inv_sh[c0 + c]);
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (c0 + c < cols) mine[(c0 + c) * D + key] = o[c];
          }
        }
        if (whole) {
          if (a.lse != nullptr && tid < cols)
            a.lse[row_sh[was][tid]] = (log2f(l_sh[tid]) - nref_sh[was][tid]) * attn::kLn2;
        } else {
          if (tid < cols) {
            mine[NQ * D + tid] = -nref_sh[was][tid];
            mine[NQ * (D + 1) + tid] = l_sh[tid];
            if (began) reinterpret_cast<long long*>(mine + NQ * (D + 2))[tid] = row_sh[was][tid];
          }
          if (began) record = make_int2(done.c_last - cta + 1, cols);
        }
      }
      if (!have) break;
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) l[c] = 0;
      const int t0 = part.t0, t1 = part.t1, n = part.n;

      for (int t = t0; t < t1; ++t, ++nt) {
        const bool first = t == t0;
        if (kAhead && t + 1 == t1) ask_q(u + 1);
        const int valid = n - t * kTile;  // keys of this tile that there are
        wait(&scale_bar[nt % kScaleSlots], nt / kScaleSlots);
        const float sv = key < valid ? scales[nt % kScaleSlots][1][key / kKv8Group] : 0.f;
        const float f = key < valid ? scales[nt % kScaleSlots][0][key / kKv8Group] : 0.f;
        wait(&s_full, nt);
        tc_fence_after();
        uint64_t x[kCols / 2];
        for (bool raised = false;; raised = true) {
          const uint64_t f2 = pack2(f, f);
          float s[kCols];
          tmem_load(tm_s, s);
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {  // x = f g S - R
            const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(&nref_sh[par][col0 + c]);
            const ulonglong2 g = *reinterpret_cast<const ulonglong2*>(&fq_sh[col0 + c]);
            x[c / 2] = fma2(pack2(s[c], s[c + 1]), mul2(f2, g.x), r.x);
            x[c / 2 + 1] = fma2(pack2(s[c + 2], s[c + 3]), mul2(f2, g.y), r.y);
          }
          if (key >= valid) {
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) x[c] = pack2(attn::neg_inf(), attn::neg_inf());
          }
          if (raised) break;
          if (!first) {
            float xm = attn::neg_inf();
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) {
              const float2 v = unpack2(x[c]);
              xm = fmaxf(xm, fmaxf(v.x, v.y));
            }
            if (!barrier_any<128>(2 + grp, attn::fast_exp2(xm) * sv > kLimit)) break;
          }
          // the largest weight x value scale of each row in this tile, as its logarithm
          const float lv = sv > 0.f ? __log2f(sv) : attn::neg_inf();
#pragma unroll
          for (int c0 = 0; c0 < kCols; c0 += 16) {  // sixteen at a time: the rare way must not cost the common one registers
            float u[16];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float2 v = unpack2(x[c0 / 2 + c]);
              u[2 * c] = v.x + lv;
              u[2 * c + 1] = v.y + lv;
            }
            const float m = reduce_transposed(u, lane, [](float p, float r) { return fmaxf(p, r); });
            if (lane < 16) red_sh[warp & 3][col0 + c0 + lane] = m;
          }
          group_sync();
          if (key < kCols) {
            const int c = col0 + key;
            const float top = fmaxf(fmaxf(red_sh[0][c], red_sh[1][c]), fmaxf(red_sh[2][c], red_sh[3][c]));
            float up = 0.f;  // what R grows by
            if ((first || top > kLimitLog2) && fabsf(top) < INFINITY) up = top - kTop;
            nref_sh[par][c] -= up;
            alpha_sh[c] = first ? 0.f : exp2f(-up);
          }
          if (!first) wait(&pv_done, nt - 1);
          group_sync();
          if (!first) {
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) l[c] = mul2(l[c], pack2(alpha_sh[col0 + 2 * c], alpha_sh[col0 + 2 * c + 1]));
#pragma unroll 1
            for (int k = 0; k < 3 * kCols / 16; ++k) {
              const int z = k % 3, c0 = k / 3 * 16;
              float o[16];
              tmem_load(tm_o + z * NQ + c0, o);
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] *= alpha_sh[col0 + c0 + c];
              tmem_store(tm_o + z * NQ + c0, o);
            }
            tmem_st_wait();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free);  // the scores are in registers
        const uint64_t sv2 = pack2(sv, sv);
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 16) {
          uint32_t part[3][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[3][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int c = c0 / 2 + 2 * j + k;
              const float2 v = unpack2(x[c]);
              const uint64_t p = pack2(attn::fast_exp2(v.x), attn::fast_exp2(v.y));
              l[c] = add2(l[c], p);
              const float2 w2 = unpack2(mul2(p, sv2));
              const uint32_t h = pack_f16x2(w2.x, w2.y);
              // e5m2 is fp16's upper byte: round to it by adding half of the lower one
              const uint32_t hi8 = (h + 0x00800080u) & 0xff00ff00u;
              const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&hi8));
              const uint32_t rb = *reinterpret_cast<const uint32_t*>(&r);
              const uint32_t mid8 = (rb + 0x00800080u) & 0xff00ff00u;
              const __half2 z = __hsub2(r, *reinterpret_cast<const __half2*>(&mid8));
              w[0][k] = hi8;
              w[1][k] = mid8;
              w[2][k] = *reinterpret_cast<const uint32_t*>(&z) + 0x00800080u;
            }
#pragma unroll
            for (int z = 0; z < 3; ++z) part[z][j] = __byte_perm(w[z][0], w[z][1], 0x7531);
          }
          if (c0 == 0 && nt > 0) wait(&pv_done, nt - 1);  // P's buffer is free
          const int chunk = (col0 + c0) / 16;
#pragma unroll
          for (int z = 0; z < 3; ++z) {
            const uint32_t at = C::kPlanes ? p_base + z * kTile * C::kPRow + swz<C::kPRow>(key, chunk)
                                           : p_base + swz<C::kPRow>(key, z * (NQ / 16) + chunk);
            st_shared_v4(at, part[z][0], part[z][1], part[z][2], part[z][3]);
          }
        }
        if (valid < kTile) {                  // what lies behind the end must not meet a weight, not even 0
          const int vi = v_index(nt);
          wait(&full_bar[vi % C::kSlots], vi / C::kSlots);
          if (tid >= valid && tid < kTile) {
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) st_shared_v4(ring + (vi % C::kSlots) * C::kSlotBytes + tid * D + i * 16, 0, 0, 0, 0);
          }
        }
        tc_fence_before();
        fence_async_smem();
        mbar_arrive(&p_ready);
      }
    }
    if (tid == 0) static_cast<int2*>(a.ws)[cta] = record;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) tmem_dealloc(tmem, C::kTmemCols);
}

// A warp joins one row of the unit that begins in piece blockIdx.x and goes on in the next ones.
constexpr int kJoinWarps = 8;

template <int D, int NQ>
__global__ void __launch_bounds__(kJoinWarps * 32) kv8_join_kernel(const Kv8AttnArgs a) {
  using C = Cfg<D, NQ>;
  constexpr int kE = D / 32, kFlight = 4;
  const int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31, cta = blockIdx.x;
  griddep_wait();
  // Three CTAs leave little of an SM's shared memory: where the next attention starts beside this kernel's blocks, which
  // hold a piece each, some SMs are left with gaps that fit two, and the last CTAs begin when the first end (about every
  // third call took 200 us for 150).  So there the next kernel starts when this one is done.
  if (C::kCtas < 3) griddep_launch_dependents();
  const float* const parts = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + kRecordBytes);
  const float* const first = parts + (static_cast<size_t>(cta) * 2 + 1) * C::kPartFloats;
  auto part = [&](int i) { return i == 0 ? first : parts + static_cast<size_t>(cta + i) * 2 * C::kPartFloats; };
  const int2 record = __ldcg(static_cast<const int2*>(a.ws) + cta);
  if (r >= record.y) return;
  const long long row = __ldcg(reinterpret_cast<const long long*>(first + NQ * (D + 2)) + r);
  float top = attn::neg_inf(), o[kE], total = 0.f;
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = 0.f;
  for (int i0 = 0; i0 < record.x; i0 += 32) {  // a piece a lane for R and l, the pieces' rows kFlight at a time
    const int n = min(32, record.x - i0);
    const float* const mine = part(i0 + min(lane, n - 1)) + NQ * D + r;
    float ref = attn::neg_inf(), sum = 0.f;
    if (lane < n) {
      ref = __ldcg(mine);
      sum = __ldcg(mine + NQ);
    }
    float w = 0.f;
    for (int j0 = 0; j0 < n; j0 += kFlight) {
      float v[kFlight][kE];
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        if (j0 + j >= n) break;
        const float* const src = part(i0 + j0 + j) + r * D + lane * kE;
        if constexpr (kE == 4)
          *reinterpret_cast<float4*>(v[j]) = __ldcg(reinterpret_cast<const float4*>(src));
        else
          *reinterpret_cast<float2*>(v[j]) = __ldcg(reinterpret_cast<const float2*>(src));
      }
      if (j0 == 0) {  // the weights, while the first rows are on their way
        float now = ref;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
        now = fmaxf(now, top);
        const float keep = exp2f(top - now);
        w = exp2f(ref - now);
        top = now;
        float add = w * sum;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) add += __shfl_xor_sync(0xffffffffu, add, d);
        total = fmaf(total, keep, add);
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] *= keep;
      }
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        if (j0 + j >= n) break;
        const float wj = __shfl_sync(0xffffffffu, w, j0 + j);
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] = fmaf(wj, v[j][e], o[e]);
      }
    }
  }
  const float inv = 1.f / total;
  __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.o) + row * D + lane * kE;
  uint32_t w[kE / 2];
#pragma unroll
  for (int e = 0; e < kE / 2; ++e) w[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  if constexpr (kE == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(out) = w[0];
  if (a.lse != nullptr && lane == 0) a.lse[row] = (top + log2f(total)) * attn::kLn2;
}

template <int D>
cudaError_t encode_codes(CUtensorMap* map, const void* ptr, uint64_t rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {D, rows};
  cuuint64_t strides[1] = {D};
  cuuint32_t box[2] = {D, kPage};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int grid_of(int nq, int num_sms) { return std::min(ctas_per_sm(nq) * num_sms, kMaxCtas); }

template <int D, int NQ>
cudaError_t launch(const Kv8AttnArgs& a, int num_sms, cudaStream_t stream) {
  using C = Cfg<D, NQ>;
  CUtensorMap tk, tv;
  const uint64_t rows = static_cast<uint64_t>(a.bt.num_pages) * a.kv.n_kv_heads * kPage;
  cudaError_t e = encode_codes<D>(&tk, a.kv.k, rows);
  if (e == cudaSuccess) e = encode_codes<D>(&tv, a.kv.v, rows);
  if (e == cudaSuccess) e = attn::set_smem(kv8_attn_kernel<D, NQ>, C::kDynSmem);
  if (e != cudaSuccess) return e;
  const int grid = grid_of(NQ, num_sms);
  e = attn::launch_pdl(kv8_attn_kernel<D, NQ>, dim3(grid), C::kThreads, C::kDynSmem, 0, stream, tk, tv, a);
  if (e != cudaSuccess || a.whole_units) return e;
  const int64_t most = static_cast<int64_t>(a.bt.max_block_len) * (a.n_heads / a.kv.n_kv_heads);
  const int joined = static_cast<int>(std::min<int64_t>(NQ, most));
  return attn::launch_pdl(kv8_join_kernel<D, NQ>, dim3(grid, (joined + kJoinWarps - 1) / kJoinWarps), kJoinWarps * 32, 0, 0,
                          stream, a);
}

// Rows that share a key head, at most: the smallest of 16, 32 and 64 that holds them, and units of 64 beyond.  A tile
// costs the softmax its NQ columns whether they are rows or not: 16 sequences with blocks of 32 take 44 us in units of
// 32, 58 in units of 64, one sequence 11.9 and 14.1.  Four rows to a key head are bound by memory either way, and 16
// leave it a little more of the SM: two contexts of 131072 keys 82.8 us in units of 16, 83.6 in units of 32 (64 single
// tokens 151 and 154).  128 rows in two units of 64 read and work on the keys twice, 43 us where the bytes take 10; a
// unit of 128, which would need one CTA an SM, was not built.
int unit_rows(int max_block_len, int n_heads, int n_kv_heads) {
  const int64_t rows = static_cast<int64_t>(max_block_len) * (n_heads / n_kv_heads);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

}  // namespace

size_t kv8_attention_workspace_bytes(int max_block_len, int n_heads, int n_kv_heads, int head_dim, int num_sms) {
  const size_t nq = unit_rows(max_block_len, n_heads, n_kv_heads);
  return kRecordBytes + static_cast<size_t>(grid_of(static_cast<int>(nq), num_sms)) * 2 * nq * (head_dim + 4) * sizeof(float);
}

cudaError_t launch_kv8_attention(const Kv8AttnArgs& args, int num_sms, cudaStream_t stream) {
  Kv8AttnArgs a = args;
  a.whole_units = a.bt.max_seq_len <= kWholeTiles * kTile ? 1 : 0;
  const int nq = unit_rows(a.bt.max_block_len, a.n_heads, a.kv.n_kv_heads);
  if (a.head_dim == 128)
    return nq == 16 ? launch<128, 16>(a, num_sms, stream)
                    : nq == 32 ? launch<128, 32>(a, num_sms, stream) : launch<128, 64>(a, num_sms, stream);
  return nq == 16 ? launch<64, 16>(a, num_sms, stream)
                  : nq == 32 ? launch<64, 32>(a, num_sms, stream) : launch<64, 64>(a, num_sms, stream);
}

}  // namespace dllm
