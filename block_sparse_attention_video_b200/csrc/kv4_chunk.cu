// kv4_chunk.cu -- attention of many query rows (chunks, prompts) over the 4-bit cache on the
// tcgen05 tensor cores: f16 operands, fp32 accumulators in tensor memory.
//
// Unit: 256 query rows of a sequence that share a KV head, as two 128-row Q tiles (slots 0
// and 1), against the pages they see, 128 keys a step; units are cut into equal pieces over
// the blocks (kv4_units.cuh). The tensor cores read f16, so the codes are expanded once per
// step for all 256 rows: what bounds the kernel is the products (4 d flops a row and key)
// and, level with them, the exponentials (one a row and key).
//
// One persistent block per SM, 512 threads (four warpgroups):
//   warps 0-3, 4-7   softmax and epilogue of slot 0 and 1 (thread = row = TMEM lane); they
//                    also bring their unit's Q rows into shared memory
//   warp  8          TMEM allocator and MMA issuer (whole warp, one elected lane issues)
//   warp  9          producer: walks the units, copies each page's K and V halves (codes and
//                    scales, 9 KB at d 128) into a ring of three
//   warps 10-15      expand the codes to f16 tiles in the 128-byte-swizzled layout of the
//                    MMA descriptors, 64 columns a half; E2M1 times E4M3 is exact in f16
// The block launches with 128 registers a thread (512 x 128 = 65,536); the softmax
// warpgroups rise to 184, the others drop to 72 (128 x 2 x (184 + 72) = 65,536).
//
// MMA order: S0(0) S1(0), then for k >= 1: PV0(k-1) S0(k) PV1(k-1) S1(k), at last PV0 PV1:
// the exponentials of one slot overlap the other slot's products. TMEM (512 columns): S0
// [0,128) S1 [128,256) O0 [256,384) O1 [384,512); P (f16, two per column) overwrites the
// first 64 columns of S and is the A operand of P.V. Shared memory: Q 2 x 32 KB, four
// expanded tiles of 32 KB (two K, two V), three raw halves.
//
// Softmax: base 2, the running max raised (and O rescaled) only when exceeded by 2^8, P
// kept at up to 2^14 of its row's reference so that f16 holds small weights too; row sums
// add the unrounded P. Q is scaled by a power of two per row, undone in the logits.
#include <cfloat>

#include "kv4_units.cuh"
#include "sm100.cuh"

namespace fvattn {
namespace kv4 {
namespace chunk {

constexpr int kThreads = 512;
constexpr int kRows = 256;
constexpr int kRegsSoftmax = 184;
constexpr int kRegsOther = 72;
constexpr int kExpand = 6;      // warps that expand codes
constexpr int kTiles = 4;       // expanded K and V tiles
constexpr int kRaw = 3;         // raw K and V halves
constexpr int kFlags = 8;       // steps whose page validity is kept: more than are in flight

template <int HD>
struct Tile {
  static constexpr int kHalves = HD / 64;
  static constexpr int kHalfBytes = 128 * 128;            // 128 rows x 64 f16 columns
  static constexpr int kBytes = kHalves * kHalfBytes;
  static constexpr int kRawBytes = kStep * (HD / 2 + HD / kGroup);
  static constexpr uint32_t kIdescQK = umma_idesc_f16(128, kStep, false);
  static constexpr uint32_t kIdescPV = umma_idesc_f16(128, HD, true);
  static constexpr int kPart = HD * 128 + 256;            // floats of one slot's partial result
};

template <int HD>
struct __align__(1024) Smem {
  uint8_t q[2][Tile<HD>::kBytes];
  uint8_t kv[kTiles][Tile<HD>::kBytes];
  uint8_t raw[kRaw][Tile<HD>::kRawBytes];
  Meta unit[2];
  uint64_t unit_full[2], unit_empty[2];
  uint64_t q_full[2];
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t kv_full[kTiles], kv_empty[kTiles];
  uint64_t s_full[2], p_full[2][2], o_full[2];
  uint64_t meet[2];
  uint64_t mma_done;
  Piece piece;
  Seqs seqs;
  int flags[kFlags];      // bit k: page k of the step is absent
  int joiner[2];
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t h;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr));
  return h;
}
__device__ __forceinline__ int lds_s32(const int* p) {
  int v;
  asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}

// ------------------------------------------------------------------ producer
template <int HD>
__device__ void produce(const AttnParams& P, Smem<HD>& sm) {
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const Entries<kRows> en(P, sm.seqs);
  const int mult = en.times();
  const int per = kStep / P.block;
  const Layout L(HD, P.block);
  const int half = L.codes + L.scales;             // K (or V) codes and scales of a page
  const long long E = en.count(), total = sm.piece.total, lo = sm.piece.lo, hi = sm.piece.hi;
  long long entry = sm.piece.entry;
  int b = 0, m0 = 0, seen = 0, which = 0, op = 0, un = 0, step = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag));
  };
  for (long long x = lo; ok;) {
    Meta m;
    m.ns = 0;
    if (x < hi) {
      int steps;
      if (x == lo) {
        steps = max(1, en.steps(entry, b, m0, seen, &m));
        which = static_cast<int>(divide(sm.piece.rem, steps, m.s0));
      } else {
        if (++which == mult) {
          which = 0;
          do ++entry; while (entry < E && en.steps(entry, b, m0, seen, nullptr) == 0);
          if (entry >= E) {                        // lengths changed under the kernel
            ok = false;
            break;
          }
        }
        steps = max(1, en.steps(entry, b, m0, seen, &m));
        m.s0 = 0;
      }
      m.h = which;
      m.m0 = m0;
      m.mc = static_cast<int>(min(static_cast<long long>(kRows), static_cast<long long>(m.q) * P.G - m0));
      m.seen = seen;
      m.ns = static_cast<int>(min(static_cast<long long>(steps - m.s0), hi - x));
      m.begin = piece_of(x - m.s0, total, sm.piece.blocks);
      m.end = piece_of(x - m.s0 + steps - 1, total, sm.piece.blocks);
    }
    const int u = un & 1;
    if (!wait(&sm.unit_empty[u], ((un >> 1) & 1) ^ 1)) { ok = false; break; }
    if (lane == 0) {
      sm.unit[u] = m;
      mbar_arrive(&sm.unit_full[u]);
    }
    ++un;
    __syncwarp();
    if (m.ns == 0) break;
    const int cnt = (seen + P.block - 1) / P.block;
    int window = -1, w_slot = -1;                  // 32 pages of the unit, one a lane
    for (int s = m.s0; ok && s < m.s0 + m.ns; ++s, ++step) {
      int slot[2] = {-1, -1};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int pos = s * per + k;
        if (k >= per || pos >= cnt) break;
        if ((pos >> 5) != window) {
          window = pos >> 5;
          const int p = window * 32 + lane;
          w_slot = p < cnt ? pool_slot(P.bt, P.c.num_pages, b, p, P.status) : -1;
        }
        slot[k] = __shfl_sync(0xffffffffu, w_slot, pos & 31);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t, ++op) {          // K, then V
        const int st = op % kRaw;
        if (!wait(&sm.raw_empty[st], ((op / kRaw) & 1) ^ 1)) { ok = false; break; }
        if (lane == 0) {
          if (t == 0) sm.flags[step % kFlags] = (slot[0] < 0 ? 1 : 0) | (slot[1] < 0 ? 2 : 0);
          const uint32_t bytes = ((slot[0] >= 0) + (slot[1] >= 0)) * half;
          if (bytes) mbar_arrive_expect_tx(&sm.raw_full[st], bytes); else mbar_arrive(&sm.raw_full[st]);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (slot[k] >= 0)
              bulk_load(sm.raw[st] + k * half,
                        P.c.pages + (static_cast<size_t>(slot[k]) * P.c.H + m.h) * L.rec + t * half, half,
                        &sm.raw_full[st]);
        }
        __syncwarp();
      }
    }
    x += m.ns;
  }
  for (int o = max(0, op - kRaw); o < op; ++o) mbar_wait_plain(&sm.raw_full[o % kRaw], (o / kRaw) & 1);
}

// ------------------------------------------------------------------ expansion to f16
// A lane expands 32 channels of a key: one 16-byte word of codes, two scales, four 16-byte
// stores. Lanes of one 8-lane phase read 128 contiguous bytes and store to eight different
// 16-byte columns of the swizzled rows (at d 128 the lanes of the second half take their
// words in the order 2 3 0 1 for that).
template <int HD>
__device__ void expand(const AttnParams& P, Smem<HD>& sm) {
  constexpr int LPR = HD / 32;                     // lanes per row
  constexpr int RPW = 32 / LPR;                    // rows per warp and pass
  const int warp = (threadIdx.x >> 5) - (16 - kExpand), lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const Layout L(HD, P.block);
  const int half = L.codes + L.scales;
  const int part = lane % LPR;
  const bool swap = part >= 2;
  const int shift = P.block == 128 ? 7 : 6;
  int op = 0, un = 0, step = 0;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag));
  };
  while (true) {
    const int u = un & 1;
    if (!wait(&sm.unit_full[u], (un >> 1) & 1)) return;
    const int ns = sm.unit[u].ns, s0 = sm.unit[u].s0, seen = sm.unit[u].seen;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.unit_empty[u]);
    ++un;
    if (ns == 0) return;
    for (int s = s0; s < s0 + ns; ++s, ++step) {
#pragma unroll 1
      for (int t = 0; t < 2; ++t, ++op) {
        const int rs = op % kRaw, ts = op % kTiles;
        if (!wait(&sm.raw_full[rs], (op / kRaw) & 1)) return;
        const int absent = lds_s32(&sm.flags[step % kFlags]);
        if (!wait(&sm.kv_empty[ts], ((op / kTiles) & 1) ^ 1)) return;
        const uint32_t raw = smem_u32(sm.raw[rs]), dst = smem_u32(sm.kv[ts]) + (part >> 1) * Tile<HD>::kHalfBytes;
        // all of the warp's rows are loaded first: the chains of conversions then overlap
        constexpr int kGroups = kStep / RPW, kRounds = (kGroups + kExpand - 1) / kExpand;
        uint32_t w[kRounds][4], sc[kRounds];
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
          if (warp + kExpand * i >= kGroups) break;
          const int row = (warp + kExpand * i) * RPW + lane / LPR;
          const int pg = row >> shift, key = row & (P.block - 1);
          const uint32_t src = raw + pg * half;
          lds128(src + key * (HD / 2) + part * 16, w[i]);
          sc[i] = lds_u16(src + L.codes + key * (HD / kGroup) + part * 2);
          // V behind the last key that a row sees, or of an absent page, is 0: memory there holds
          // anything, and P = 0 times NaN would not be 0
          if (t == 1 && (s * kStep + row >= seen || ((absent >> pg) & 1))) sc[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
          if (warp + kExpand * i >= kGroups) break;
          const int row = (warp + kExpand * i) * RPW + lane / LPR;
          const __half2 hs = e4m3x2_to_half2(sc[i]);
          const uint32_t h = *reinterpret_cast<const uint32_t*>(&hs);
          const uint32_t f[2] = {__byte_perm(h, 0, swap ? 0x3232 : 0x1010), __byte_perm(h, 0, swap ? 0x1010 : 0x3232)};
          const uint32_t words[4] = {swap ? w[i][2] : w[i][0], swap ? w[i][3] : w[i][1], swap ? w[i][0] : w[i][2],
                                     swap ? w[i][1] : w[i][3]};
          const uint32_t base = dst + row * 128;
          const int c0 = (part & 1) * 4, r7 = row & 7;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t v[4];
            e2m1x8_to_half2(words[y], v);
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] = mul2(v[z], f[y >> 1]);
            sts128(base + (((c0 + (swap ? (y ^ 2) : y)) ^ r7) * 16), v);
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.kv_full[ts]);
          mbar_arrive(&sm.raw_empty[rs]);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ MMA issue
template <int HD>
__device__ void issue(const AttnParams& P, Smem<HD>& sm, uint32_t tmem) {
  using T = Tile<HD>;
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const uint64_t dq[2] = {umma_desc_sw128(smem_u32(sm.q[0]), 16, 1024), umma_desc_sw128(smem_u32(sm.q[1]), 16, 1024)};
  const uint64_t dk = umma_desc_sw128(smem_u32(sm.kv[0]), 16, 1024);
  const uint64_t dv = umma_desc_sw128(smem_u32(sm.kv[0]), T::kHalfBytes, 1024);
  int base = 0, un = 0, qn[2] = {0, 0}, pn[2] = {0, 0};
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag));
  };
  bool ok = true;
  while (ok) {
    const int u = un & 1;
    if (!wait(&sm.unit_full[u], (un >> 1) & 1)) break;
    const int ns = *reinterpret_cast<volatile int*>(&sm.unit[u].ns);
    const bool two = *reinterpret_cast<volatile int*>(&sm.unit[u].mc) > 128;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.unit_empty[u]);
    ++un;
    if (ns == 0) break;
    auto ready = [&](int o) -> bool { return wait(&sm.kv_full[o % kTiles], (o / kTiles) & 1); };
    auto s_op = [&](int X, int k) -> bool {          // S_X = Q_X K(k)^T
      if (k == 0) {
        if (!wait(&sm.q_full[X], qn[X] & 1)) return false;
        ++qn[X];
      }
      tc_fence_after();
      const uint64_t ks = dk + static_cast<uint64_t>(((base + 2 * k) % kTiles) * (T::kBytes >> 4));
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t o = ((kk >> 2) * T::kHalfBytes + (kk & 3) * 32) >> 4;
        umma_ss_elect(tmem + X * 128, dq[X] + o, ks + o, T::kIdescQK, kk > 0 ? 1u : 0u);
      }
      umma_commit_elect(&sm.s_full[X]);
      return true;
    };
    auto pv_op = [&](int X, int k) -> bool {         // O_X += P_X V(k), P in two halves of 64 keys
      const uint64_t vs = dv + static_cast<uint64_t>(((base + 2 * k + 1) % kTiles) * (T::kBytes >> 4));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!wait(&sm.p_full[X][h], pn[X] & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = h * 4; kk < h * 4 + 4; ++kk)
          umma_ts_elect(tmem + 256 + X * 128, tmem + X * 128 + kk * 8, vs + static_cast<uint32_t>((kk * 16 * 128) >> 4),
                        T::kIdescPV, (k > 0 || kk > 0) ? 1u : 0u);
      }
      ++pn[X];
      return true;
    };
    ok = ready(base) && s_op(0, 0) && (!two || s_op(1, 0));
    if (ok) umma_commit_elect(&sm.kv_empty[base % kTiles]);
    for (int k = 1; ok && k < ns; ++k) {
      ok = ready(base + 2 * k - 1) && pv_op(0, k - 1) && ready(base + 2 * k) && s_op(0, k) && (!two || pv_op(1, k - 1));
      if (!ok) break;
      umma_commit_elect(&sm.kv_empty[(base + 2 * k - 1) % kTiles]);
      ok = !two || s_op(1, k);
      if (!ok) break;
      umma_commit_elect(&sm.kv_empty[(base + 2 * k) % kTiles]);
    }
    if (ok) ok = ready(base + 2 * ns - 1) && pv_op(0, ns - 1) && (!two || pv_op(1, ns - 1));
    if (ok) {
      umma_commit_elect(&sm.kv_empty[(base + 2 * ns - 1) % kTiles]);
      umma_commit_elect(&sm.o_full[0]);
      if (two) umma_commit_elect(&sm.o_full[1]);
    }
    base += 2 * ns;
  }
  // every MMA issued has completed before TMEM is freed
  umma_commit_elect(&sm.mma_done);
  mbar_wait_plain(&sm.mma_done, 0);
}

// ------------------------------------------------------------------ softmax and epilogue
template <int HD>
__device__ void softmax(const AttnParams& P, Smem<HD>& sm, uint32_t tmem) {
  using T = Tile<HD>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const int X = warp >> 2, quad = warp & 3;
  const int row = quad * 32 + lane;                  // row of the slot
  const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t tS = tmem + lane_off + X * 128, tO = tmem + lane_off + 256 + X * 128;
  int un = 0, sn = 0, on = 0, step = 0, met = 0;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag));
  };
#pragma unroll 1
  while (true) {
    const int u = un & 1;
    if (!wait(&sm.unit_full[u], (un >> 1) & 1)) return;
    const Meta& m = sm.unit[u];                      // kept until the unit's end, read again there
    const int ns = m.ns;
    if (ns == 0 || X * 128 >= m.mc) {                // no unit, or no rows in this slot: warp-uniform
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[u]);
      ++un;
      if (ns == 0) return;
      step += ns;
      continue;
    }
    ++un;
    // this thread's row of the call's tensors and query head
    auto place = [&](int& i_row, int& head) -> bool {
      const int rr = X * 128 + row;
      const bool live = rr < m.mc;
      i_row = live ? (m.m0 + rr) / P.G : 0;
      head = m.h * P.G + (live ? (m.m0 + rr) - i_row * P.G : 0);
      return live;
    };
    float cs;                                        // logits per unit of S
    int left;                                        // keys that the row sees from this step on
    // ---- Q: this thread's row, scaled so that its largest element lies in [2^13, 2^14)
    {
      int i_row, head, ex = 0;
      const bool live = place(i_row, head);
      uint4 w[HD / 8];
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.q) +
                                                        static_cast<long long>(m.cu + i_row) * P.q_stride + head * HD);
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        w[i] = live ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
          mx = fmax3(mx, fabsf(__uint_as_float(v[y] << 16)), fabsf(__uint_as_float(v[y] & 0xFFFF0000u)));
      }
      if (mx > 0.f && mx <= FLT_MAX) ex = min(13 - ilogbf(mx), 126);
      const float f1 = exp2f(static_cast<float>(ex / 2)), f2 = exp2f(static_cast<float>(ex - ex / 2));
      const uint32_t dst = smem_u32(sm.q[X]) + row * 128;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t p[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          p[y] = pack_f16(__uint_as_float(v[y] << 16) * f1 * f2, __uint_as_float(v[y] & 0xFFFF0000u) * f1 * f2);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + (i >> 3) * T::kHalfBytes +
                                                                      (((i & 7) ^ (row & 7)) * 16)),
                     "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3])
                     : "memory");
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[X]);
      const float base = P.scale_log2 * (P.c.k_scale ? __ldg(P.c.k_scale + m.h) : 1.f);
      // never 0, so that a masked key's -inf stays -inf
      cs = fmaxf(base * exp2f(static_cast<float>(-(ex / 2))) * exp2f(static_cast<float>(-(ex - ex / 2))), FLT_MIN);
      const int n = m.n;
      left = (live ? (P.causal ? min(max(m.start + i_row + 1, 0), n) : n) : 0) - m.s0 * kStep;
    }
    float mref = kFloor, l_run = 0.f;
#pragma unroll 1
    for (int k = 0; k < ns; ++k, ++step, left -= kStep) {
      if (!wait(&sm.s_full[X], sn & 1)) return;
      ++sn;
      tc_fence_after();
      const int absent = lds_s32(&sm.flags[step % kFlags]) & (kStep / P.block == 2 ? 3 : 1);
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
      tmem_wait_ld();
      if (__any_sync(0xffffffffu, left < kStep || absent != 0)) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool gone = (absent >> (c * 32 / P.block)) & 1;
          const int v = gone ? 0 : left - c * 32;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i >= v) s[c][i] = __float_as_uint(-INFINITY);
        }
      }
      float mx8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) mx8[i] = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          mx8[i & 7] = fmax3(mx8[i & 7], __uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1]));
      const float mx =
          fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])) * cs;
      const bool need = mx > mref + (kHead + kRaise);
      if (k == 0) {
        mref = fmaxf(mx - kHead, kFloor);            // O is not yet there
      } else if (__any_sync(0xffffffffu, need)) {    // vote: the TMEM accesses below take the whole warp
        const float nm = need ? mx - kHead : mref;
        const float f = ex2_approx(mref - nm);
        l_run *= f;
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st32(tO + c * 32, o);
        }
        tmem_wait_st();
        mref = nm;
      }
      const float2 c2 = make_float2(cs, cs), negm = make_float2(-mref, -mref);
      float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x =
              __ffma2_rn(make_float2(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), c2, negm);
          const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
          ls[i & 1] = __fadd2_rn(ls[i & 1], make_float2(p0, p1));
          pk[i] = pack_f16(p0, p1);
        }
        tmem_st16(tS + c * 16, pk);
        if (c & 1) {                                 // a half of P is complete
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[X][c >> 1]);
        }
      }
      l_run += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
    }
    // ---- epilogue
    if (!wait(&sm.o_full[X], on & 1)) return;
    ++on;
    tc_fence_after();
    int i_row, head;
    const bool live = place(i_row, head);
    const int begin = m.begin, end = m.end;
    const float vs = P.c.v_scale ? __ldg(P.c.v_scale + m.h) : 1.f;
    const size_t at = static_cast<size_t>(m.cu + i_row) * P.c.H * P.G + head;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.unit_empty[u]);
    __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(P.out) + at * HD;
    if (begin == end) {
      const float inv = l_run > 0.f || l_run != l_run ? vs / l_run : 0.f;
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + c * 32, o);
        tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              w[y] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * y]) * inv, __uint_as_float(o[8 * i + 2 * y + 1]) * inv);
            reinterpret_cast<uint4*>(orow)[c * 4 + i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (live && P.lse) P.lse[at] = l_run > 0.f || l_run != l_run ? (mref + log2f(l_run)) * kLn2 : -INFINITY;
      tc_fence_before();
      continue;
    }
    // The unit lies in blocks begin .. end: O to the workspace ([HD/4][128] float4, a row a
    // thread), and who finds all parts there joins them in the order of the blocks.
    auto part_of = [&](int i) {
      return P.part + ((static_cast<size_t>(i) * 2 + (i == begin ? 1 : 0)) * 2 + X) * T::kPart;
    };
    {
      float* mine = part_of(blockIdx.x);
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + c * 32, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          reinterpret_cast<uint4*>(mine)[(c * 8 + i) * 128 + row] =
              make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
      mine[HD * 128 + row] = mref;
      mine[HD * 128 + 128 + row] = l_run;
    }
    tc_fence_before();
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.meet[X]);
      return wait(&sm.meet[X], met++ & 1);
    };
    if (!meet()) return;
    if (quad == 0) {   // one warp's fences, between the barriers, cover the slot's stores and loads
      const bool all = leave_part(P.left, P.status.call, begin, end,
                                  [&](int i) { return (2 * i + (i == begin ? 1 : 0)) * 2 + X; });
      if (lane == 0) sm.joiner[X] = all;
    }
    if (!meet()) return;
    if (!sm.joiner[X]) continue;
    float mx = kFloor, sum = 0.f;
    for (int i = begin; i <= end; ++i) mx = fmaxf(mx, __ldcg(part_of(i) + HD * 128 + row));
    for (int i = begin; i <= end; ++i) {
      const float* p = part_of(i) + HD * 128;
      sum = fmaf(__ldcg(p + 128 + row), ex2_approx(__ldcg(p + row) - mx), sum);
    }
    const float inv = sum > 0.f || sum != sum ? vs / sum : 0.f;
#pragma unroll 1
    for (int c = 0; c < HD / 32; ++c) {
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = begin; i <= end; ++i) {
        const float* p = part_of(i);
        const float f = ex2_approx(__ldcg(p + HD * 128 + row) - mx) * inv;
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const float4 a = __ldcg(reinterpret_cast<const float4*>(p) + (c * 8 + y) * 128 + row);
          v[y].x = fmaf(a.x, f, v[y].x); v[y].y = fmaf(a.y, f, v[y].y);
          v[y].z = fmaf(a.z, f, v[y].z); v[y].w = fmaf(a.w, f, v[y].w);
        }
      }
      if (live) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          reinterpret_cast<uint4*>(orow)[c * 4 + i] =
              make_uint4(pack_bf16x2(v[2 * i].x, v[2 * i].y), pack_bf16x2(v[2 * i].z, v[2 * i].w),
                         pack_bf16x2(v[2 * i + 1].x, v[2 * i + 1].y), pack_bf16x2(v[2 * i + 1].z, v[2 * i + 1].w));
      }
    }
    if (live && P.lse) P.lse[at] = sum > 0.f || sum != sum ? (mx + log2f(sum)) * kLn2 : -INFINITY;
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) attn_chunk_kernel(const AttnParams P) {
  extern __shared__ uint8_t smem_raw[];
  Smem<HD>& sm = *reinterpret_cast<Smem<HD>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.unit_full[i], 1);
      mbar_init(&sm.unit_empty[i], 9 + kExpand);   // 8 softmax warps, the issuer, those that expand
      mbar_init(&sm.q_full[i], 4);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], 4);
      mbar_init(&sm.p_full[i][1], 4);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.meet[i], 4);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&sm.raw_full[i], 1);
      mbar_init(&sm.raw_empty[i], kExpand);
    }
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&sm.kv_full[i], kExpand);
      mbar_init(&sm.kv_empty[i], 1);
    }
    mbar_init(&sm.mma_done, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
  }
  // A unit's own costs (Q, epilogue) are about three steps'.
  find_piece<kRows, kThreads>(P, sm.seqs, sm.piece, 4);
  if (sm.piece.hi <= sm.piece.lo) return;    // block-uniform, nothing allocated yet
  if (warp == 8) {                           // whole warp
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  // All threads meet here once at the end (every wait before it is bounded); then the
  // allocating warp frees TMEM. Each role has its own copy, for its own register limit.
  auto teardown = [&]() {
    __syncwarp();
    tc_fence_before();
    asm volatile("barrier.sync 1, %0;" ::"n"(kThreads) : "memory");
    if (warp == 8) {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem, 512);
      if ((threadIdx.x & 31) == 0 && sm.abort_flag) record_status(P.status, FVATTN_ERR_TIMEOUT);
    }
  };
  if (warp >= 8) {
    regs_dec<kRegsOther>();
    if (warp == 8) issue<HD>(P, sm, tmem);
    else if (warp == 9) produce<HD>(P, sm);
    else expand<HD>(P, sm);
    teardown();
    return;
  }
  regs_inc<kRegsSoftmax>();
  softmax<HD>(P, sm, tmem);
  teardown();
}

template <int HD>
static cudaError_t launch(const AttnParams& P, int grid, cudaStream_t st) {
  const int smem = static_cast<int>(sizeof(Smem<HD>)) + 1024;
  cudaError_t e = cudaFuncSetAttribute(attn_chunk_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_chunk_kernel<HD><<<grid, kThreads, smem, st>>>(P);
  return cudaGetLastError();
}

}  // namespace chunk

size_t chunk_part_bytes(int d, int grid) { return static_cast<size_t>(grid) * 4 * (d * 128 + 256) * sizeof(float); }

cudaError_t launch_chunk(const AttnParams& P, int d, int grid, cudaStream_t st) {
  return d == 128 ? chunk::launch<128>(P, grid, st) : chunk::launch<64>(P, grid, st);
}

}  // namespace kv4
}  // namespace fvattn
