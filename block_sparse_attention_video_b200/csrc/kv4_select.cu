// kv4_select.cu -- the pages a row attends: softmax over the mean keys of the full
// pages before the row's own, averaged over the query heads of a KV head, then Top-p
// with a Top-k floor.
//
// All arithmetic is fp64: the page sums are exact integers and q is exact, so a score
// differs from its definition by a few 2^-53 and only true ties are decided by rounding.
//
// One block per group of rows of a sequence and KV head. Up to eight (row, query head)
// pairs share every page's sum, which is converted to fp64 once for all of them. The floor of
// a call of many rows is the fp64 units (d multiply-adds a pair and page, 64 a clock and
// SM), of single tokens HBM (4 d bytes a page); what bounds both is the latency of one
// block's chain (780 rows over 591 pages: a sixth look-up, two fifths scores, a sixth softmax, a
// third search and list), so loads go out several at a time and, in large grids, three blocks
// share an SM.
//   1. scores: fp64 tensor products of 8 pairs x 8 pages x 4 channels. q lies in shared memory;
//      a page's sums are loaded straight into the operand's lanes (the order of channels in
//      a dot product is free: lane t of a quad takes channels 16 i + 4 t .. + 3, 16 bytes).
//   2. softmax of each pair over its pages and the mean over a row's pairs, in shared memory.
//   3. per row one warp finds the smallest mass v* whose pages and those above reach p:
//      a bracket of values is narrowed until at most 32 masses are left, which it sorts.
//      Pages tied at v* are taken in index order. If the floor is larger, the k_min-th mass
//      is found the same way on counts.
#include "kv4_units.cuh"

namespace fvattn {
namespace kv4 {

constexpr int kSelThreads = 256;
constexpr int kAtOnce = 4;     // masses a lane loads before it looks at the first
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

struct SelectParams {
  Cache c;
  Batch bt;
  const void* q;
  long long q_stride;
  int G, RU, pairs;       // query heads per KV head; rows and (row, head) pairs per block
  double w;               // scale / (1024 block)
  float p;
  int k_min, block, stride;   // stride: scores per row in shared memory (max_pages, whole tiles of 8)
  int* kv_idx;
  int* kv_cnt;
  Status status;
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 32 values, one a lane, in descending order.
__device__ __forceinline__ double sort32(double v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const double u = __shfl_xor_sync(0xffffffffu, v, stride);
      const bool first = (lane & stride) == 0, desc = (lane & size) == 0;
      v = first == desc ? fmax(v, u) : fmin(v, u);
    }
  return v;
}

// What the search of a row's cut finds: the mass v*, the number of pages selected and of those
// above v*.
struct Cut {
  double star;
  int cnt, above;
};

// The cut among at most 32 masses, one a lane, v descending: those above them number c_hi and
// sum to f_hi. False if no prefix reaches p.
__device__ __forceinline__ bool cut_sorted(double v, int in, int c_hi, double f_hi, double target, Cut& cut) {
  const int lane = threadIdx.x & 31;
  double sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  const unsigned reach = __ballot_sync(0xffffffffu, f_hi + sum >= target && lane < in);
  if (reach == 0u) return false;
  const int at = __ffs(reach) - 1;
  cut.star = __shfl_sync(0xffffffffu, v, at);
  cut.cnt = c_hi + at + 1;
  cut.above = c_hi + __popc(__ballot_sync(0xffffffffu, v > cut.star));
  return true;
}

// Puts the masses of a bracket one after the other: `m` is this lane's mass of 32, `in` whether it
// belongs, `have` how many there are already; `box` holds 32.
__device__ __forceinline__ void gather32(double m, bool in, double* box, int& have) {
  const unsigned ins = __ballot_sync(0xffffffffu, in);
  const int k = have + __popc(ins & ((1u << (threadIdx.x & 31)) - 1u));
  if (in && k < 32) box[k] = m;
  have += __popc(ins);
}
// This lane's one of the gathered masses, 0 behind the last.
__device__ __forceinline__ double gathered(const double* box, int have) {
  __syncwarp();
  const int lane = threadIdx.x & 31;
  const double v = lane < have ? box[lane] : 0.0;
  __syncwarp();
  return v;
}

// The cut, found in two stages. fp32 copies f of the masses narrow a bracket of values until at
// most 32 masses are in it; a probe moves an end only where the fp32 sum is 2^-16 from p or
// more (the sum of n <= 8192 rounded masses of total 1 is off by less than (n/32 + 7) 2^-24 <
// 2^-15.9 at the worst and n / 2^29 as a rule; what it decides is checked in fp64). The masses
// above the bracket are then added, and those inside sorted and added, in fp64. False if that
// does not settle it.
__device__ bool quick_cut(const double* x, const float* f, int n, float p, double* box, Cut& cut) {
  const int lane = threadIdx.x & 31;
  constexpr float kClear = 0x1p-16f;
  float mx = 0.f;
#pragma unroll 4
  for (int j = lane; j < n; j += 32) mx = fmaxf(mx, f[j]);
  // What lies below v* and v* itself sum to more than 1 - p: v* > (1 - p) / n.
  unsigned lo = __float_as_uint((1.f - p) / n * 0.99f);
  unsigned hi = __reduce_max_sync(0xffffffffu, __float_as_uint(mx)) + 1u;
  int c_lo = n, c_hi = 0;                    // c_lo: an upper bound until a probe has moved lo
  while (c_lo - c_hi > 32) {
    if (hi <= lo + 1u) return false;
    // three probes a pass, at the quarters: a pass waits for its loads and reductions
    const unsigned quarter = (hi - lo) >> 2, mid[3] = {lo + quarter, lo + ((hi - lo) >> 1), hi - max(quarter, 1u)};
    float a[3] = {0.f, 0.f, 0.f};
    int c[3] = {0, 0, 0};
#pragma unroll 4
    for (int j = lane; j < n; j += 32) {
      const float m = f[j];
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        const bool ge = m >= __uint_as_float(mid[u]);
        a[u] += ge ? m : 0.f;
        c[u] += ge ? 1 : 0;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < 3; ++u) a[u] += __shfl_xor_sync(0xffffffffu, a[u], o);
    const unsigned lo0 = lo, hi0 = hi;
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      c[u] = __reduce_add_sync(0xffffffffu, c[u]);
      if (a[u] >= p + kClear) { lo = mid[u]; c_lo = c[u]; }
      else if (a[u] < p - kClear && hi == hi0) { hi = mid[u]; c_hi = c[u]; }
    }
    if (lo == lo0 && hi == hi0) return false;
  }
  const float vlo = __uint_as_float(lo), vhi = __uint_as_float(hi);
  double above = 0.0;
  int have = 0;
#pragma unroll 1
  for (int j0 = 0; j0 < n; j0 += 32 * kAtOnce) {
    float m[kAtOnce];
    double d[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int j = j0 + 32 * u + lane;
      m[u] = j < n ? f[j] : -1.f;
      d[u] = j < n ? x[j] : 0.0;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      above += m[u] >= vhi ? d[u] : 0.0;
      gather32(d[u], m[u] >= vlo && m[u] < vhi, box, have);
    }
  }
  above = warp_sum(above);
  const double target = static_cast<double>(p);
  if (have > 32 || above >= target) return false;
  return cut_sorted(sort32(gathered(box, have)), have, c_hi, above, target, cut);
}

// The same for any n and any masses, in fp64 throughout: bisection of the bit patterns of
// non-negative doubles. F(v) = the sum of the masses >= v, added up in a fixed order, falls
// as v rises. by_count: the cut at `want` masses instead of at the sum p. False if no prefix
// reaches p.
__device__ bool full_cut(const double* x, int n, double target, bool by_count, int want, double* box, Cut& cut) {
  using u64 = unsigned long long;
  const int lane = threadIdx.x & 31;
  auto bits_of = [](double v) { return static_cast<u64>(__double_as_longlong(v)); };
  auto value_of = [](u64 b) { return __longlong_as_double(static_cast<long long>(b)); };
  auto measure = [&](u64 bits, double& F, int& C) {
    const double v = value_of(bits);
    double a = 0.0;
    int c = 0;
    for (int j = lane; j < n; j += 32) {
      const double m = x[j];
      if (m >= v) {
        a += m;
        ++c;
      }
    }
    F = warp_sum(a);
    C = __reduce_add_sync(0xffffffffu, c);
  };
  double mx = 0.0;
  for (int j = lane; j < n; j += 32) mx = fmax(mx, x[j]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  // bracket [lo, hi): c_lo masses at or above lo, c_hi (of sum f_hi) at or above hi
  u64 lo = 0, hi = bits_of(mx) + 1;
  int c_lo = n, c_hi = 0;
  double F, f_hi = 0.0;
  if (!by_count) {
    measure(0, F, c_lo);
    if (!(F >= target)) return false;
  }
  while (c_lo - c_hi > 32 && hi - lo > 1) {
    const u64 mid = lo + ((hi - lo) >> 1);
    int C;
    measure(mid, F, C);
    if (by_count ? C >= want : F >= target) { lo = mid; c_lo = C; } else { hi = mid; c_hi = C; f_hi = F; }
  }
  if (c_lo - c_hi > 32) {                    // equal masses, taken one by one
    cut.star = value_of(lo);
    int need = 1;
    double acc = f_hi + cut.star;
    while (acc < target && need < c_lo - c_hi) { acc += cut.star; ++need; }
    cut.cnt = by_count ? want : c_hi + need;
    cut.above = c_hi;
    return true;
  }
  int have = 0;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    const double m = j < n ? x[j] : 0.0;
    gather32(m, j < n && bits_of(m) >= lo && bits_of(m) < hi, box, have);
  }
  const double v = sort32(gathered(box, have));
  if (by_count) {
    cut.star = __shfl_sync(0xffffffffu, v, want - c_hi - 1);
    cut.cnt = want;
    cut.above = c_hi + __popc(__ballot_sync(0xffffffffu, v > cut.star));
    return true;
  }
  return cut_sorted(v, have, c_hi, f_hi, target, cut);
}

// Top-p with the floor on masses x[0..n), n >= 1: the selected pages ascending, then n itself.
// Whole warp; every value that steers it is the same in all lanes.
__device__ void pick_pages(const double* x, const float* f, int n, float p, int k_min, double* box, int* out,
                           int* out_cnt) {
  const int lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1u;
  Cut cut;
  bool all = p >= 1.f || k_min >= n;
  if (!all) {
    bool found = quick_cut(x, f, n, p, box, cut);
    if (!found) found = full_cut(x, n, static_cast<double>(p), false, 0, box, cut);
    all = !found;
    if (found && cut.cnt < k_min) full_cut(x, n, 2.0, true, k_min, box, cut);   // the floor
  }
  // all pages above v*, and at v* the first ones that fill the count
  const int take = all ? 0 : cut.cnt - cut.above;
  int written = 0, tied = 0;
  // (masses are not negative, so their bit patterns compare as they do; 64-bit float compares wait
  // for the fp64 units. Where a mass is a NaN, all pages are taken.)
  const long long star = all ? 0 : __double_as_longlong(cut.star);
#pragma unroll 1
  for (int j0 = 0; j0 < n; j0 += 32 * kAtOnce) {
    long long m[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int j = j0 + 32 * u + lane;
      m[u] = j < n ? __double_as_longlong(x[j]) : -1ll;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int j = j0 + 32 * u + lane;
      const bool eq = !all && m[u] == star;
      const unsigned eqs = __ballot_sync(0xffffffffu, eq);
      const bool sel = j < n && (all || m[u] > star || (eq && tied + __popc(eqs & below) < take));
      const unsigned sels = __ballot_sync(0xffffffffu, sel);
      if (sel) out[written + __popc(sels & below)] = j;
      written += __popc(sels);
      tied += __popc(eqs);
    }
  }
  if (lane == 0) {
    out[written] = n;
    *out_cnt = written + 1;
  }
}

// C[8 x 8] += A[8 x 4] B[4 x 8] in fp64; a lane holds A[lane/4][lane%4], B[lane%4][lane/4] and
// C[lane/4][2 (lane%4)], C[lane/4][2 (lane%4) + 1].
__device__ __forceinline__ void mma_f64(double (&c)[2], double a, double b) {
  asm("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
      : "+d"(c[0]), "+d"(c[1])
      : "d"(a), "d"(b));
}

// Three blocks share an SM (kThree) or two, which then have the registers to fetch ahead.
template <typename T, int HD, bool kThree>
__global__ void __launch_bounds__(kSelThreads, kThree ? 3 : 2) select_kernel(const SelectParams P) {
  constexpr int PAIRS = 8, kWarps = kSelThreads / 32;
  static_assert(PAIRS == kWarps, "a warp brings a pair's q");
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ __align__(16) double qs[PAIRS][HD + 2];   // two off: the quads' reads take all banks
  __shared__ double scale[PAIRS];                      // 1 / (sum of a pair's exponentials * G)
  __shared__ double box[kWarps][32];
  __shared__ Seqs seqs;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = P.G, RU = P.RU, NP = P.pairs, LD = P.stride;
  double* xs = reinterpret_cast<double*>(raw);                       // [NP][LD] scores
  double* mass = G == 1 ? xs : xs + static_cast<size_t>(NP) * LD;    // [RU][LD]
  float* fmass = reinterpret_cast<float*>(xs + static_cast<size_t>(NP + (G == 1 ? 0 : RU)) * LD);   // [RU][LD]
  int* slots = reinterpret_cast<int*>(fmass + static_cast<size_t>(RU) * LD);                        // [LD]
  open_call(P.status);
  seqs.load<kSelThreads>(P.bt);
  __syncthreads();
  const int *cu = seqs.rows_of(P.bt), *kv_len = seqs.lengths_of(P.bt);
  check_rows(P.bt, cu, P.status);
  // Groups are numbered without a prefix sum: sequence b owns those from cu[b]/RU + b on.
  const int h = blockIdx.x % P.c.H, tile = blockIdx.x / P.c.H;
  int lo = 0, hi = P.bt.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] / RU + mid <= tile) lo = mid; else hi = mid;
  }
  const int b = lo, r0 = cu[b], r1 = cu[b + 1];
  const int first = r0 + (tile - (r0 / RU + b)) * RU;                // first row of the group
  const int rows = min(RU, min(r1, rows_end(P.bt, cu)) - first);
  if (r0 < 0 || first < r0 || rows <= 0) return;
  const int n = held(kv_len[b], P.bt, P.block, P.status);
  const int pos0 = start_of(kv_len[b], r1 - first);                  // position of the first row
  const int last = min(pos0 + rows, n) - 1;                          // last position of the group
  const int most = last < 0 ? 0 : last / P.block;                    // pages to score
  const double w = P.w * (P.c.k_scale ? static_cast<double>(__ldg(P.c.k_scale + h)) : 1.0);
  const int chunks = (G + NP - 1) / NP;                              // of query heads; one if RU > 1
  // Pages that row i of the group scores; 0 for a row outside the sequence (recorded below).
  auto own_of = [&](int i) { return i < rows && pos0 + i >= 0 && pos0 + i < n ? (pos0 + i) / P.block : 0; };
  for (int ch = 0; ch < chunks; ++ch) {
    // pair k: row k / G, head k % G (RU rows), or head ch * NP + k of the one row
    auto row_of = [&](int k) { return RU > 1 ? k / G : 0; };
    auto head_of = [&](int k) { return RU > 1 ? k % G : ch * NP + k; };
    auto live = [&](int k) { return k < NP && row_of(k) < rows && (RU > 1 ? k < RU * G : head_of(k) < G); };
    // a warp brings a pair's q; the pool slots are looked up while it is on its way
    struct alignas(sizeof(T) * HD / 32) Part { T x[HD / 32]; } part;
    const bool here = live(warp);
    if (here)
      part = *reinterpret_cast<const Part*>(static_cast<const T*>(P.q) +
                                            static_cast<long long>(first + row_of(warp)) * P.q_stride +
                                            (static_cast<long long>(h) * G + head_of(warp)) * HD + lane * (HD / 32));
    if (ch == 0)
      for (int j = tid; j < most; j += kSelThreads) slots[j] = pool_slot(P.bt, P.c.num_pages, b, j, P.status);
#pragma unroll
    for (int i = 0; i < HD / 32; ++i)
      qs[warp][lane * (HD / 32) + i] = here ? static_cast<double>(to_float(part.x[i])) : 0.0;
    __syncthreads();
    // ---- scores: 8 pairs x 8 pages a warp and tile; a lane's channels are 16 i + 4 t .. + 3.
    // With two blocks an SM the next tile's sums are on their way while this one's are multiplied.
    {
      const int g = lane >> 2, t = lane & 3;
      const int* sums = P.c.ksum + static_cast<size_t>(h) * HD + 4 * t;
      const size_t page = static_cast<size_t>(P.c.H) * HD;
      int4 v[HD / 16];
      auto fetch = [&](int j0) {
        const int slot = j0 + g < most ? slots[j0 + g] : 0;
        const int4* k4 = reinterpret_cast<const int4*>(sums + max(slot, 0) * page);
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) v[i] = __ldg(k4 + 4 * i);
      };
      if (!kThree && warp * 8 < most) fetch(warp * 8);
#pragma unroll 1
      for (int j0 = warp * 8; j0 < most; j0 += kWarps * 8) {
        int4 u[HD / 16];
        if (kThree) fetch(j0);
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) u[i] = v[i];
        if (!kThree && j0 + kWarps * 8 < most) fetch(j0 + kWarps * 8);
        double c[2][2] = {{0.0, 0.0}, {0.0, 0.0}};                   // two chains
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          const double2 a0 = *reinterpret_cast<const double2*>(&qs[g][16 * i + 4 * t]);
          const double2 a1 = *reinterpret_cast<const double2*>(&qs[g][16 * i + 4 * t + 2]);
          mma_f64(c[0], a0.x, static_cast<double>(u[i].x));
          mma_f64(c[1], a0.y, static_cast<double>(u[i].y));
          mma_f64(c[0], a1.x, static_cast<double>(u[i].z));
          mma_f64(c[1], a1.y, static_cast<double>(u[i].w));
        }
        // An invalid page (recorded; some page's sums were read in its place) scores 0. The row of
        // scores and the slots are padded to whole tiles.
        const int2 from = *reinterpret_cast<const int2*>(&slots[j0 + 2 * t]);
        if (g < NP)
          *reinterpret_cast<double2*>(&xs[static_cast<size_t>(g) * LD + j0 + 2 * t]) =
              make_double2(from.x >= 0 ? (c[0][0] + c[1][0]) * w : 0.0, from.y >= 0 ? (c[0][1] + c[1][1]) * w : 0.0);
      }
    }
    __syncthreads();
    // ---- softmax of each pair over the pages before its row's own: a warp per pair
    if (warp < NP) {
      const int own = live(warp) ? own_of(row_of(warp)) : 0;
      double* x = xs + static_cast<size_t>(warp) * LD;
      double mx = -INFINITY, z = 0.0;
#pragma unroll 4
      for (int j = lane; j < own; j += 32) mx = fmax(mx, x[j]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
#pragma unroll 4
      for (int j = lane; j < own; j += 32) {
        const double e = exp(x[j] - mx);
        x[j] = e;
        z += e;
      }
      z = warp_sum(z);
      z = z > 0.0 ? 1.0 / (z * G) : 0.0;
      if (G == 1) {                                                  // the pair's row: x is its masses' place
#pragma unroll 4
        for (int j = lane; j < own; j += 32) {
          const double m = x[j] * z;
          x[j] = m;
          fmass[static_cast<size_t>(warp) * LD + j] = static_cast<float>(m);
        }
      } else if (lane == 0) {
        scale[warp] = z;
      }
    }
    __syncthreads();
    if (G == 1) break;
    // ---- mean over the heads of each row
    const int per = RU > 1 ? G : min(NP, G - ch * NP);               // pairs of a row in this chunk
#pragma unroll 1
    for (int i = 0; i < rows; ++i) {
      const int own = own_of(i);
      const double* x = xs + static_cast<size_t>(i) * per * LD;
      for (int j = tid; j < own; j += kSelThreads) {
        double m = ch > 0 ? mass[static_cast<size_t>(i) * LD + j] : 0.0;
        for (int k = 0; k < per; ++k) m = fma(x[static_cast<size_t>(k) * LD + j], scale[i * per + k], m);
        mass[static_cast<size_t>(i) * LD + j] = m;
        fmass[static_cast<size_t>(i) * LD + j] = static_cast<float>(m);
      }
    }
    __syncthreads();
  }
  // ---- one warp per row
  for (int i = warp; i < rows; i += kWarps) {
    const size_t unit = static_cast<size_t>(first + i) * P.c.H + h;
    int* out = P.kv_idx + unit * P.bt.max_pages;
    const int own = own_of(i);
    if (own == 0) {
      if (lane == 0) {
        const bool outside = pos0 + i < 0 || pos0 + i >= n;
        if (outside) record_status(P.status, FVATTN_ERR_INVALID_ARG); else out[0] = 0;
        P.kv_cnt[unit] = outside ? 0 : 1;
      }
      continue;
    }
    pick_pages(mass + static_cast<size_t>(i) * LD, fmass + static_cast<size_t>(i) * LD, own, P.p, P.k_min, box[warp],
               out, P.kv_cnt + unit);
  }
}

// Shared memory of the scores, the masses (fp64 and fp32) and the pool slots.
static size_t select_smem(int pairs, int ru, int G, int stride) {
  return static_cast<size_t>(pairs + (G == 1 ? 0 : ru)) * stride * sizeof(double) +
         static_cast<size_t>(ru + 1) * stride * sizeof(float);
}

template <typename T, int HD>
static cudaError_t select_t(SelectParams& P, cudaStream_t st) {
  // Up to eight (row, head) pairs a block, as shared memory holds them beside 13 KB of fixed
  // size: eight up to 2,000 pages, down to one at 8,192.
  P.pairs = 8;
  while (P.pairs > 1 && select_smem(P.pairs, P.pairs > P.G ? P.pairs / P.G : 1, P.G, P.stride) > 208 * 1024) P.pairs /= 2;
  P.RU = P.pairs > P.G ? P.pairs / P.G : 1;
  if (P.RU == 1) P.pairs = min(P.pairs, P.G);
  const long long grid = (static_cast<long long>(P.bt.rows) / P.RU + P.bt.B) * P.c.H;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const int smem = static_cast<int>(select_smem(P.pairs, P.RU, P.G, P.stride));
  // Three blocks an SM, where they fit and the rows fill more than two on each of 148 SMs: 1,176
  // blocks of 591 pages 130 us, 136 with two that fetch ahead; 256 blocks of 512 pages 30 and 25 us.
  const bool three = static_cast<long long>(P.bt.rows) / P.RU * P.c.H > 2 * 148 && smem <= 62 * 1024;
  auto kernel = three ? select_kernel<T, HD, true> : select_kernel<T, HD, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(grid), kSelThreads, smem, st>>>(P);
  return cudaGetLastError();
}

cudaError_t launch_select(const Cache& c, const Batch& bt, const void* q, long long q_stride, int Hq, bool bf16,
                          float scale, float p, int k_min, int d, int block, int* kv_idx, int* kv_cnt,
                          const Status& status, cudaStream_t st) {
  SelectParams P;
  P.c = c;
  P.bt = bt;
  P.q = q;
  P.q_stride = q_stride;
  P.G = Hq / c.H;
  P.RU = P.pairs = 1;
  P.w = static_cast<double>(scale) / (1024.0 * block);
  P.p = p;
  P.k_min = k_min;
  P.block = block;
  P.stride = (bt.max_pages + 7) & ~7;
  P.kv_idx = kv_idx;
  P.kv_cnt = kv_cnt;
  P.status = status;
  if (d == 128) return bf16 ? select_t<__nv_bfloat16, 128>(P, st) : select_t<float, 128>(P, st);
  return bf16 ? select_t<__nv_bfloat16, 64>(P, st) : select_t<float, 64>(P, st);
}

}  // namespace kv4
}  // namespace fvattn
