// kv4_units.cuh -- how the attention kernels of the 4-bit cache divide their work.
//
// Unit: up to RT query rows (a sequence's (row, query head) pairs that share a KV head, in
// that order; with lists, the query heads of one row) against the pages they see. A step is
// 128 keys: one page of 128 tokens or two of 64. The steps of all units form one line that is
// cut into equal pieces, one per block, so ragged and causal lengths balance by themselves:
// every block adds up the units' lengths and finds its piece. A unit that lies in several
// pieces leaves partial sums in the workspace; the block that finds them all there joins them in
// the order of the pieces, so the result does not depend on who that is.
#pragma once

#include "kv4.cuh"
#include "sm100.cuh"

namespace fvattn {
namespace kv4 {

constexpr int kStep = 128;                          // keys per step
constexpr float kFloor = -3.0e38f;                  // running max before any key
constexpr float kRaise = 8.f;                       // the max is raised when exceeded by 2^8
constexpr float kHead = 6.f;                        // P <= 2^(6 + 8) stays inside fp16
constexpr float kLn2 = 0.69314718055994531f;

// mbar_wait of sm100.cuh without a status word: bounded, false on abort. A wait that runs out
// raises the abort flag; who sees that at its end records FVATTN_ERR_TIMEOUT.
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(a, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
      *abort_flag = 1;
      return false;
    }
  }
}

struct AttnParams {
  Cache c;
  Batch bt;
  const void* q;
  long long q_stride;
  void* out;
  float* lse;
  const int* kv_idx;      // nullptr: every page
  const int* kv_cnt;
  float scale_log2;       // scale * log2(e)
  int G, causal, block;
  Status status;
  unsigned long long* left;      // flags of the parts left in `part`: the number of the call that left them
  float* part;            // partial results of units that lie in several blocks
};

// A unit, as its producer publishes it to the other warps.
struct alignas(16) Meta {
  int cu, q, n;           // the sequence: first row, rows (of the tensors), tokens held
  int start;              // position of its first row
  int m0, mc;             // first (row, head) pair and their number
  int h;                  // KV head
  int seen;               // keys that the unit's last row sees
  int begin, end;         // blocks that hold the unit's first and last step
  int s0, ns;             // first of the unit's steps in this block, and their number
};

// First rows and lengths of the sequences, copied to shared memory where they are few: the
// searches below are chains of loads.
struct Seqs {
  static constexpr int kMax = 256;
  int cu[kMax + 1];
  int kv_len[kMax];
  __device__ const int* rows_of(const Batch& bt) const { return bt.B <= kMax ? cu : bt.cu; }
  __device__ const int* lengths_of(const Batch& bt) const { return bt.B <= kMax ? kv_len : bt.kv_len; }
  template <int kThreads>
  __device__ void load(const Batch& bt) {
    if (bt.B > kMax) return;
    for (int i = threadIdx.x; i <= bt.B; i += kThreads) {
      cu[i] = __ldg(bt.cu + i);
      if (i < bt.B) kv_len[i] = __ldg(bt.kv_len + i);
    }
  }
};

// a / b and the remainder for a >= 0, b > 0: 32-bit where both fit.
__device__ __forceinline__ long long divide(long long a, int b, int& rest) {
  if (a <= 0xFFFFFFFFll) {
    const unsigned q = static_cast<unsigned>(a) / static_cast<unsigned>(b);
    rest = static_cast<int>(static_cast<unsigned>(a) - q * b);
    return q;
  }
  const long long q = a / b;
  rest = static_cast<int>(a - q * b);
  return q;
}

// Entries are what the units are counted by: without lists, tiles of RT pairs of a
// sequence (each counts for all KV heads); with lists, (row, KV head) (each counts for
// all tiles of its query heads). Tiles are numbered without a prefix sum: sequence b owns
// those from cu[b] G / RT + b on, room for the at most ceil(q G / RT) it needs.
template <int RT>
struct Entries {
  const AttnParams& P;
  const int* cu;          // shared memory or global
  const int* kv_len;
  __device__ Entries(const AttnParams& p, const Seqs& s)
      : P(p), cu(s.rows_of(p.bt)), kv_len(s.lengths_of(p.bt)) {}
  __device__ long long count() const {
    return P.kv_idx ? static_cast<long long>(P.bt.rows) * P.c.H
                    : static_cast<long long>(P.bt.rows) * P.G / RT + P.bt.B;
  }
  // start_of, at most the table's end: a row there or behind it sees every token held.
  __device__ int start(int n, int q) const { return min(start_of(n, q), P.bt.max_pages * P.block); }
  __device__ int times() const { return P.kv_idx ? (P.G + RT - 1) / RT : P.c.H; }
  // Steps of a unit of entry e and where it lies; 0 if the entry is not in use.
  __device__ int steps(long long e, int& b, int& m0, int& seen, Meta* m) const {
    if (P.kv_idx) {
      int cnt = __ldg(P.kv_cnt + e);
      int h;
      const int r = static_cast<int>(divide(e, P.c.H, h));
      if (r >= cu[P.bt.B]) return 0;
      int lo = 0, hi = P.bt.B;                  // cu[lo] <= r < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= r) lo = mid; else hi = mid;
      }
      b = lo;
      if (cu[b] < 0 || r < cu[b]) return 0;     // skipped (r - cu[b] has no bound), or before the first
      if (cnt < 0 || cnt > P.bt.max_pages) {
        record_status(P.status, FVATTN_ERR_INVALID_ARG);
        cnt = min(max(cnt, 0), P.bt.max_pages);
      }
      m0 = (r - cu[b]) * P.G;
      if (m) {
        m->cu = cu[b];
        m->q = cu[b + 1] - m->cu;
        m->n = held(kv_len[b], P.bt, P.block, P.status);
        m->start = start(kv_len[b], m->q);
        const int pos = m->start + (r - m->cu);
        seen = P.causal ? min(max(pos + 1, 0), m->n) : m->n;
      }
      return max(1, (cnt * P.block + kStep - 1) / kStep);
    }
    int lo = 0, hi = P.bt.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (static_cast<long long>(cu[mid]) * P.G / RT + mid <= e) lo = mid; else hi = mid;
    }
    b = lo;
    const int r0 = cu[b], r1 = cu[b + 1];
    const int q = min(r1, rows_end(P.bt, cu)) - r0;
    const long long first = (e - (static_cast<long long>(r0) * P.G / RT + b)) * RT;
    if (r0 < 0 || q <= 0 || first < 0 || first >= static_cast<long long>(q) * P.G) return 0;
    m0 = static_cast<int>(first);
    const int n = held(kv_len[b], P.bt, P.block, P.status);
    const int last = min((m0 + RT - 1) / P.G, q - 1);
    const int pos0 = start(kv_len[b], r1 - r0);
    seen = P.causal ? min(max(pos0 + last + 1, 0), n) : n;
    if (m) {
      m->cu = r0;
      m->q = q;
      m->n = n;
      m->start = pos0;
    }
    return max(1, (seen + kStep - 1) / kStep);
  }
};

// The block's piece [lo, hi) of the line of steps, and the entry and offset of lo.
struct Piece {
  long long warp_total[32];
  long long lo, hi, rem, total;
  int entry, blocks;
};

// Called by all threads of the block (has block barriers); at least `least` steps go to a
// block that gets any.
template <int RT, int kThreads>
__device__ void find_piece(const AttnParams& P, Seqs& seqs, Piece& sm, int least) {
  open_call(P.status);
  seqs.load<kThreads>(P.bt);
  __syncthreads();
  const Entries<RT> en(P, seqs);
  check_rows(P.bt, en.cu, P.status);
  const long long E = en.count();
  const int mult = en.times();
  const long long chunk = (E + kThreads - 1) / kThreads;
  const long long e0 = min(E, threadIdx.x * chunk), e1 = min(E, e0 + chunk);
  int b, m0, seen;
  long long mine = 0;
  for (long long e = e0; e < e1; ++e) mine += static_cast<long long>(en.steps(e, b, m0, seen, nullptr)) * mult;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm.warp_total[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm.warp_total[w];
    total += sm.warp_total[w];
  }
  const long long blocks = max(1ll, min(static_cast<long long>(gridDim.x), (total + least - 1) / least));
  const long long i = blockIdx.x;
  const long long lo = i < blocks ? total * i / blocks : total;
  const long long hi = i < blocks ? total * (i + 1) / blocks : total;
  if (threadIdx.x == 0) {
    sm.lo = lo;
    sm.hi = hi;
    sm.total = total;
    sm.blocks = static_cast<int>(blocks);
  }
  long long at = before + incl - mine;
  if (lo >= at && lo < at + mine) {
    for (long long e = e0; e < e1; ++e) {
      const long long n = static_cast<long long>(en.steps(e, b, m0, seen, nullptr)) * mult;
      if (lo < at + n) {
        sm.entry = static_cast<int>(e);
        sm.rem = lo - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
}

// Marks a block's part of a unit as left, and tells whether all parts of the unit are: flags[at(i)]
// for i in begin .. end, each the number of the call that left the part. Whole warp, after a barrier
// that orders the block's stores of the part. Every block stores its flag before it looks at the
// others' (sequentially consistent fences between), so the last one to store sees them all; should
// another see them too, both join the same parts to the same result. No counter is incremented:
// nothing has to be reset, and blocks do not queue for one word.
template <typename At>
__device__ __forceinline__ bool leave_part(unsigned long long* flags, unsigned long long call, int begin, int end,
                                           At&& at) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(flags + at(static_cast<int>(blockIdx.x))), "l"(call)
                 : "memory");
    asm volatile("fence.sc.gpu;" ::: "memory");
  }
  __syncwarp();
  bool all = true;
  for (int i = begin + lane; i <= end; i += 32) {
    unsigned long long f;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(f) : "l"(flags + at(i)) : "memory");
    all = all && f == call;
  }
  return __all_sync(0xffffffffu, all);
}

// Block that holds position x of the line: the largest i with floor(total i / blocks) <= x,
// that is total i < (x + 1) blocks. An estimate, corrected with products: 64-bit divisions
// cost hundreds of cycles here.
__device__ __forceinline__ int piece_of(long long x, long long total, int blocks) {
  const long long limit = (x + 1) * blocks;
  int i = static_cast<int>(static_cast<float>(x) * (static_cast<float>(blocks) / static_cast<float>(total)));
  i = min(max(i, 0), blocks - 1);
  while (i > 0 && total * i >= limit) --i;
  while (i + 1 < blocks && total * (i + 1) < limit) ++i;
  return i;
}

}  // namespace kv4
}  // namespace fvattn
