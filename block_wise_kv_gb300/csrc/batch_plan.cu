// batch_plan.cu — the batch from request lengths, on the device, in one launch.
//
// Per sequence b: need_b = ceil(N_b / 64), take_b = max(0, need_b - held_b),
// give_b = max(0, held_b - need_b).  Four exclusive sums over the batch (block
// rows, sequence rows, pages taken, pages given) place everything else.
//
// Every CTA scans the whole batch itself (12 to 16 bytes a sequence, from L2),
// a chunk of kChunk sequences at a time, and then does its share of the chunk's
// rows and moved pages: no CTA waits for another and there is no second launch.
// That works in place because what is read is never written: pages are taken
// from the ring's head and given back behind its tail, table entries below
// held_b are only read and those from held_b on only written (or, where there was no
// page for them, looked at by the one thread that clears them), and a row in a page that
// this call hands out takes the id from the ring, not from the table.
//
// Bound: a step's plan is latency (a chain of two dependent loads and one block
// scan: 64 sequences 5.7 us); a plan of many prompts is the 12 bytes a row of the
// three row maps behind that (512 prompts of 2.1 M rows 12.7 us; 392 with one row to a
// thread, which searched the sums for each).
#include <algorithm>

#include "attn_common.cuh"
#include "kv8.cuh"

namespace dllm {
namespace {

constexpr int kThreads = 512;
constexpr int kCtasPerSm = 2;
constexpr int kChunk = kThreads;  // sequences scanned at a time, one a thread
constexpr int kWarps = kThreads / 32;

struct Sums {
  long long rows, seq, take, give;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.rows + b.rows, a.seq + b.seq, a.take + b.take, a.give + b.give};
}
__device__ __forceinline__ Sums shfl_up(const Sums& v, int d) {
  return {__shfl_up_sync(0xffffffffu, v.rows, d), __shfl_up_sync(0xffffffffu, v.seq, d),
          __shfl_up_sync(0xffffffffu, v.take, d), __shfl_up_sync(0xffffffffu, v.give, d)};
}

struct Chunk {
  long long row0[kChunk], take0[kChunk], give0[kChunk];  // exclusive sums over the whole batch
  int start[kChunk], held[kChunk], now[kChunk];          // block start, pages held before and after
};

// The largest i < n with v[i] <= x (v is increasing, v[0] <= x).
__device__ __forceinline__ int last_not_above(const long long* v, int n, long long x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Those of the four entries of a row map from j0 (a multiple of 4) on that lie in [lo, hi).
__device__ __forceinline__ void store4(int32_t* map, long long j0, const int (&v)[4], long long lo, long long hi) {
  if (map == nullptr) return;
  if (j0 >= lo && j0 + 4 <= hi) {
    *reinterpret_cast<int4*>(map + j0) = make_int4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (j0 + e >= lo && j0 + e < hi) map[j0 + e] = v[e];
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) batch_plan_kernel(const PlanArgs a) {
  __shared__ Chunk c;
  __shared__ Sums warp_sums[kWarps + 1];
  __shared__ int warp_granted[kWarps];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int cta = blockIdx.x, n_cta = gridDim.x;
  griddep_wait();

  const long long first = static_cast<long long>(cta) * kThreads + t, stride = static_cast<long long>(n_cta) * kThreads;
  int head = a.state[0], count = a.state[1];
  int err = 0;
  if (head < 0 || head >= a.num_pages || count < 0 || count > a.num_pages) {
    err |= kErrBadShape;
    head = count = 0;
  }
  auto ring_at = [&](long long i) {  // slot of the i-th id from the head on, i < 2 num_pages
    long long s = head + i;
    while (s >= a.num_pages) s -= a.num_pages;
    return static_cast<int>(s);
  };
  auto ring_id = [&](long long i) {
    const int id = a.ring[ring_at(i)];
    if (id >= 0 && id < a.num_pages) return id;
    err |= kErrBadPage;
    return -1;
  };

  Sums carry = {0, 0, 0, 0};
  int granted = 0;  // pages handed out up to and including this thread's last sequence that got some
  for (int b0 = 0; b0 < a.batch; b0 += kChunk) {
    const int b = b0 + t;
    Sums mine = {0, 0, 0, 0};
    int held = 0, start = 0, need = 0;
    bool bad_held = false;
    if (b < a.batch) {
      int n = a.seq_len[b], rows = a.block_len[b];
      start = a.block_start[b];
      held = a.held[b];
      bad_held = held < 0 || held > a.max_pages;
      const bool bad_n = n < 0 || n > a.max_seq_len;
      if (bad_held || bad_n) {  // the sequence keeps its pages, its lengths count as 0
        err |= kErrBadShape;
        n = rows = start = 0;
      }
      need = (bad_held || bad_n) ? held : (n + kPage - 1) / kPage;
      if (rows < 0 || start < 0 || rows > n - start) {
        if (rows < 0 || (rows > 0 && n > 0)) err |= kErrBadShape;  // (a length of 0 is a place without a request: no rows)
        rows = 0;
      }
      mine = {rows, n, bad_held || need < held ? 0 : need - held, bad_held || need > held ? 0 : held - need};
    }
    Sums incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums o = shfl_up(incl, d);
      if (lane >= d) incl = incl + o;
    }
    __syncthreads();  // the previous chunk's readers are done
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      const Sums w = lane < kWarps ? warp_sums[lane] : Sums{0, 0, 0, 0};
      Sums s = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const Sums o = shfl_up(s, d);
        if (lane >= d) s = s + o;
      }
      if (lane < kWarps) warp_sums[lane] = {s.rows - w.rows, s.seq - w.seq, s.take - w.take, s.give - w.give};
      if (lane == 31) warp_sums[kWarps] = s;
    }
    __syncthreads();
    const Sums at = {carry.rows + warp_sums[warp].rows + incl.rows - mine.rows,
                     carry.seq + warp_sums[warp].seq + incl.seq - mine.seq,
                     carry.take + warp_sums[warp].take + incl.take - mine.take,
                     carry.give + warp_sums[warp].give + incl.give - mine.give};
    const bool short_of = mine.take > 0 && at.take + mine.take > count;
    if (short_of) err |= kErrNoPages;
    const int now = short_of ? held : need;
    c.row0[t] = at.rows;
    c.take0[t] = at.take;
    c.give0[t] = at.give;
    c.start[t] = start;
    c.held[t] = held;
    c.now[t] = now;
    if (cta == 0 && b < a.batch) {
      a.cu_block[b] = static_cast<int>(min(at.rows, static_cast<long long>(INT32_MAX)));
      a.cu_seq[b] = static_cast<int>(min(at.seq, static_cast<long long>(INT32_MAX)));
      a.held_out[b] = now;
    }
    if (mine.take > 0 && !short_of) granted = static_cast<int>(at.take + mine.take);
    __syncthreads();
    const Sums total = carry + warp_sums[kWarps];
    const int nb = min(kChunk, a.batch - b0);

    // the ids handed out, and those given back: CTA c has every n_cta-th stretch of kThreads of this chunk's
    for (long long i = carry.take + first; i < total.take; i += stride) {
      const int k = last_not_above(c.take0, nb, i);
      int32_t* const entry = a.table + static_cast<size_t>(b0 + k) * a.max_pages + c.held[k] + (i - c.take0[k]);
      if (c.now[k] > c.held[k])
        *entry = ring_id(i);
      else if (*entry >= 0 && *entry < a.num_pages)  // asked for more than was free: a page named here may be another's by now
        *entry = -1;
    }
    for (long long i = carry.give + first; i < total.give; i += stride) {
      const int k = last_not_above(c.give0, nb, i);
      int id = a.table[static_cast<size_t>(b0 + k) * a.max_pages + c.now[k] + (i - c.give0[k])];
      if (id < 0 || id >= a.num_pages) {
        err |= kErrBadPage;
        id = -1;
      }
      if (count + i >= a.num_pages) {  // more pages than there are: the ring's live part stays as it is
        err |= kErrBadShape;
        continue;
      }
      a.ring[ring_at(count + i)] = id;
    }
    // the rows: four in a row to a thread, one search for all, 16-byte stores where all four are of this chunk
    const long long row_end = min(total.rows, static_cast<long long>(a.cap_rows));
    for (long long j0 = carry.rows / 4 * 4 + 4 * first; j0 < row_end; j0 += 4 * stride) {
      int k = last_not_above(c.row0, nb, max(j0, carry.rows));
      int slot[4], seq[4], pos[4];
      int at = -1, base = -1;  // the last page looked up (sequence k's page at): its first slot
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const long long j = j0 + e;
        slot[e] = seq[e] = pos[e] = -1;
        if (j < carry.rows || j >= row_end) continue;
        while (k + 1 < nb && c.row0[k + 1] <= j) {
          ++k;
          at = -1;
        }
        const int p = c.start[k] + static_cast<int>(j - c.row0[k]), pg = p / kPage;
        seq[e] = b0 + k;
        pos[e] = p;
        if (a.row_slot == nullptr) continue;
        if (pg != at) {
          at = pg;
          base = -1;
          if (pg < c.now[k]) {
            const int id = pg < c.held[k] ? a.table[static_cast<size_t>(b0 + k) * a.max_pages + pg]
                                          : ring_id(c.take0[k] + pg - c.held[k]);
            if (id >= 0 && id < a.num_pages)
              base = id * kPage;
            else
              err |= kErrBadPage;
          }
        }
        slot[e] = base < 0 ? -1 : base + p % kPage;
      }
      store4(a.row_slot, j0, slot, carry.rows, row_end);
      store4(a.row_seq, j0, seq, carry.rows, row_end);
      store4(a.row_pos, j0, pos, carry.rows, row_end);
    }
    carry = total;
  }
  if (cta == 0) {
    // the asked-for sums only grow, so what was handed out ends with the last sequence that got pages
    for (int d = 16; d > 0; d >>= 1) granted = max(granted, __shfl_xor_sync(0xffffffffu, granted, d));
    if (lane == 0) warp_granted[warp] = granted;
    __syncthreads();
    if (t == 0) {
      for (int w = 1; w < kWarps; ++w) granted = max(granted, warp_granted[w]);
      a.cu_block[a.batch] = static_cast<int>(min(carry.rows, static_cast<long long>(INT32_MAX)));
      a.cu_seq[a.batch] = static_cast<int>(min(carry.seq, static_cast<long long>(INT32_MAX)));
      a.state_out[0] = ring_at(granted);
      a.state_out[1] = static_cast<int>(min(static_cast<long long>(count) - granted + carry.give,
                                            static_cast<long long>(a.num_pages)));
    }
  }
  if (carry.rows > a.cap_rows || carry.seq > a.cap_seq) err |= kErrBadShape;
  for (long long j = carry.rows + first; j < a.cap_rows; j += stride) {
    if (a.row_slot != nullptr) a.row_slot[j] = -1;
    if (a.row_seq != nullptr) a.row_seq[j] = -1;
    if (a.row_pos != nullptr) a.row_pos[j] = -1;
  }
  if (err) report_error(a.err, err);
}

}  // namespace

cudaError_t launch_batch_plan(const PlanArgs& a, int num_sms, cudaStream_t stream) {
  // One CTA for each 4096 rows or pages that may have to be written, at most two an SM: each CTA repeats
  // the scan, so more of them only pay where there is enough to write (512 prompts of 2.1 M rows: 12.7 us, 1692 with one
  // CTA; 64 sequences of 32 rows take one CTA, 5.7 us, as with one for each 512).
  const long long pages = static_cast<long long>(a.batch) * a.max_pages;
  const long long most = std::max<long long>(a.cap_rows, std::min<long long>(pages, a.num_pages));
  const int grid = static_cast<int>(std::max(1ll, std::min(static_cast<long long>(kCtasPerSm * num_sms), most / 4096)));
  return attn::launch_pdl(batch_plan_kernel, dim3(grid), kThreads, 0, 0, stream, a);
}

}  // namespace dllm
