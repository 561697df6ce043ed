// kv4_attn.cu -- attention of few query rows over the 4-bit cache: single tokens,
// drafts, selected pages, and every fp32 call. One pass over the cache with the running
// maximum and sum of the softmax, split over the pages and joined in a fixed order.
//
// Units of up to 8 NT query rows, cut into equal pieces over the blocks (kv4_units.cuh).
//
// A block is one producer warp, which brings whole page records into a ring of shared
// memory (one bulk copy a page, 18 KB at d 128), and four consumer warps with 32 keys of
// the step each, as two tiles of 16 whose chains of instructions overlap. What bounds it is HBM: d + d/8 bytes of K and V a token and KV head.
//
// Arithmetic per tile, on m16n8k16 fp16 products with fp32 sums:
//   S^T [16 keys x 8 rows]     = K [16 x d] Q^T      K's codes become fp16 in registers
//   O^T [16 channels x 8 rows] += V^T [16 x 16 keys] P^T
// The transposed forms put keys (channels) on the 16-wide side and the few query rows on
// the 8-wide one. Both operands come out of shared memory as 4-bit codes and are expanded
// in registers; E2M1 times E4M3 needs at most 6 significant bits, so the fp16 operands
// hold the stored values exactly. The order of channels inside a dot product and of keys
// inside a sum is free, and is chosen so that a lane reads whole 16-byte (K) and 8-byte
// (V) words of the plain record: k-slot j of lane t is channel (HD/4) t + 4 j.., row g of
// V's tile i is channel (HD/8) g + 2 i. P^T's registers are S^T's transposed
// (movmatrix).
//
// Q is scaled by a power of two per row so that its largest element lies in [2^13, 2^14)
// (undone in the logits), so bf16 enters exactly. fp32 Q and P are split into two fp16
// parts, and O is then summed outside the tensor core, whose sums are cut off and not
// rounded.
#include <cfloat>

#include "kv4_units.cuh"
#include "sm100.cuh"

namespace fvattn {
namespace kv4 {

constexpr int kConsumers = 4;                       // consumer warps
constexpr int kTiles = 2;                           // tiles of 16 keys a warp and step
constexpr int kThreads = (kConsumers + 1) * 32;
// Steps a block takes at least: joining costs about as much. (One of the fp32 path's, which
// take three times as long.)
constexpr int kLeast = 4;
static_assert(kStep == kConsumers * kTiles * 16, "");

template <int HD, int NT>
struct Shape {
  static constexpr int RT = 8 * NT;
  static constexpr int kStageBytes = kStep * (HD + HD / 8);
  // three blocks on an SM with 55 KB of ring each; two with 74 KB beside the larger sums of NT 2
  static constexpr int kStages = (NT == 1 ? 3 : 4) * (128 / HD);
  static constexpr int kPart = RT * HD + 2 * RT;    // floats of a partial result
};

template <int HD, int NT>
struct __align__(128) AttnSmem {
  using S = Shape<HD, NT>;
  uint8_t ring[S::kStages][S::kStageBytes];
  float slab[kConsumers][S::RT][HD + 2];
  float mx[2][kConsumers][S::RT];
  float sum[2][kConsumers][S::RT];
  int4 step[S::kStages];  // first keys of the stage's two pages (-1: no such page), -, unit ends here
  Meta unit[2];
  uint64_t unit_full[2], unit_empty[2];
  uint64_t full[S::kStages];
  uint64_t empty[S::kStages];
  uint64_t sync;
  Piece piece;
  Seqs seqs;
  int joiner;
  int abort_flag;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8x8 matrix of 16-bit elements, one 32-bit row piece a lane, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint32_t x) { return __half22float2(*reinterpret_cast<__half2*>(&x)); }
__device__ __forceinline__ uint32_t e4m3x2(uint32_t two_codes) {
  const __half2 h = e4m3x2_to_half2(two_codes);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Bounded wait of a whole warp; one poll and a vote when the phase is there already.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const Status& status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) return true;
  if (__all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag))) return true;
  if ((threadIdx.x & 31) == 0) record_status(status, FVATTN_ERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }

// The producer warp: walks the piece's units, publishes each before its pages, and keeps
// the ring full.
template <int HD, int NT>
__device__ void produce(const AttnParams& P, AttnSmem<HD, NT>& sm) {
  using S = Shape<HD, NT>;
  constexpr int RT = S::RT;
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const Entries<RT> en(P, sm.seqs);
  const long long E = en.count();
  const int mult = en.times();
  const int per = kStep / P.block;                 // pages per step
  const int rec = Layout(HD, P.block).rec;
  const long long total = sm.piece.total, lo = sm.piece.lo, hi = sm.piece.hi;
  long long entry = sm.piece.entry;
  Meta m;
  int b = 0, m0 = 0, seen = 0, steps = 0, which = 0, it = 0, un = 0;
  bool ok = true;
  for (long long x = lo; ok && x < hi; x += m.ns) {
    m.s0 = 0;
    if (x == lo) {
      steps = max(1, en.steps(entry, b, m0, seen, &m));
      which = static_cast<int>(divide(sm.piece.rem, steps, m.s0));
    } else if (++which == mult) {
      which = 0;
      do ++entry; while (entry < E && (steps = en.steps(entry, b, m0, seen, &m)) == 0);
      if (entry >= E) {                            // lengths changed under the kernel
        ok = false;
        break;
      }
    }
    int cnt;                                       // pages of the unit
    if (P.kv_idx) {
      divide(entry, P.c.H, m.h);
      m.m0 = m0 + which * RT;
      m.mc = min(RT, P.G - which * RT);
      cnt = min(max(__ldg(P.kv_cnt + entry), 0), P.bt.max_pages);
    } else {
      m.h = which;
      m.m0 = m0;
      m.mc = static_cast<int>(
          min(static_cast<long long>(RT), static_cast<long long>(m.q) * P.G - m0));
      cnt = (seen + P.block - 1) / P.block;
    }
    m.seen = seen;
    m.ns = static_cast<int>(min(static_cast<long long>(steps - m.s0), hi - x));
    m.begin = x - m.s0 >= lo ? static_cast<int>(blockIdx.x) : piece_of(x - m.s0, total, sm.piece.blocks);
    m.end = x - m.s0 + steps <= hi ? static_cast<int>(blockIdx.x) : piece_of(x - m.s0 + steps - 1, total, sm.piece.blocks);
    // Pool slots of 32 pages of the unit at a time, one a lane, and the first key of each.
    int window = (m.s0 * per) >> 5, w_slot = -1, w_key = -1;
    auto look_up = [&]() {
      const int p = window * 32 + lane;
      w_slot = w_key = -1;
      if (p >= cnt) return;
      int page = p;
      if (P.kv_idx) {
        const int* list = P.kv_idx + entry * P.bt.max_pages;
        page = __ldg(list + p);
        const int before = p ? __ldg(list + p - 1) : -1;
        if (page < 0 || static_cast<long long>(page) * P.block >= m.n || (p && page <= before)) {
          record_status(P.status, FVATTN_ERR_INVALID_ARG);
          return;
        }
        if (page * P.block >= seen) return;
      }
      w_slot = pool_slot(P.bt, P.c.num_pages, b, page, P.status);
      if (w_slot >= 0) w_key = page * P.block;
    };
    const int u = un & 1;
    if (!warp_wait(&sm.unit_empty[u], ((un >> 1) & 1) ^ 1, abort_flag, P.status)) { ok = false; break; }
    ++un;
    if (lane == 0) {
      sm.unit[u] = m;
      mbar_arrive(&sm.unit_full[u]);
    }
    look_up();
    const uint8_t* pool = P.c.pages + static_cast<size_t>(m.h) * rec;
    const size_t slot_bytes = static_cast<size_t>(P.c.H) * rec;
    for (int s = m.s0; s < m.s0 + m.ns; ++s, ++it) {
      const int pos = s * per;                     // the pages of a step share a window
      if ((pos >> 5) != window) {
        window = pos >> 5;
        look_up();
      }
      const int slot0 = __shfl_sync(0xffffffffu, w_slot, pos & 31), key0 = __shfl_sync(0xffffffffu, w_key, pos & 31);
      int slot1 = __shfl_sync(0xffffffffu, w_slot, (pos + 1) & 31), key1 = __shfl_sync(0xffffffffu, w_key, (pos + 1) & 31);
      if (per == 1) slot1 = key1 = -1;
      const int st = it % S::kStages;
      if (!warp_wait(&sm.empty[st], ((it / S::kStages) & 1) ^ 1, abort_flag, P.status)) { ok = false; break; }
      if (lane == 0) {
        sm.step[st] = make_int4(key0, key1, 0, s + 1 == m.s0 + m.ns);
        const uint32_t bytes = ((slot0 >= 0) + (slot1 >= 0)) * rec;
        if (bytes) mbar_arrive_expect_tx(&sm.full[st], bytes); else mbar_arrive(&sm.full[st]);
        if (slot0 >= 0) bulk_load(sm.ring[st], pool + slot0 * slot_bytes, rec, &sm.full[st]);
        if (slot1 >= 0) bulk_load(sm.ring[st] + rec, pool + slot1 * slot_bytes, rec, &sm.full[st]);
      }
      __syncwarp();
    }
  }
  // every copy has landed before the block may end
  for (int o = max(0, it - S::kStages); o < it; ++o) mbar_wait_plain(&sm.full[o % S::kStages], (o / S::kStages) & 1);
}

template <typename T, int HD, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : sizeof(T) == 4 ? 1 : 2)
    attn_stream_kernel(const AttnParams P) {
  using S = Shape<HD, NT>;
  constexpr int RT = S::RT;
  constexpr bool kExact = sizeof(T) == 4;          // fp32: operands in two fp16 parts
  constexpr int KS = HD / 16;                      // k-steps of S, and 16-channel tiles of O
  constexpr int KW = HD / 32;                      // 32-bit words of K a lane and key
  // 16-byte alignment is all that the copies need; the struct sits at the start as it is, so
  // that every access is known to be to shared memory
  extern __shared__ __align__(128) uint8_t smem_raw[];
  AttnSmem<HD, NT>& sm = *reinterpret_cast<AttnSmem<HD, NT>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kConsumers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.unit_full[i], 1);
      mbar_init(&sm.unit_empty[i], kConsumers);
    }
    mbar_init(&sm.sync, kConsumers);
    sm.abort_flag = 0;
    fence_mbarrier_init();
  }
  find_piece<RT, kThreads>(P, sm.seqs, sm.piece, kExact ? 1 : kLeast);
  const int len = static_cast<int>(sm.piece.hi - sm.piece.lo);
  if (len <= 0) return;
  if (warp == kConsumers) {
    produce<HD, NT>(P, sm);
    return;
  }

  // ------------------------------------------------------------------ consumers
  // All consumers meet here; bounded like every wait of the library, so that a lost
  // warp cannot hold the others for good.
  int met = 0;
  auto meet = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.sync);
    return warp_wait(&sm.sync, met++ & 1, abort_flag, P.status);
  };
  const int g = lane >> 2, t = lane & 3;
  // Row g of a tile is the tile's key g ^ (g>>1 & 1): neighbouring lanes' V rows then lie
  // in different halves of the banks.
  const int gk = g ^ ((g >> 1) & 1);
  const int ka = (2 * t) ^ (t & 1), kb = (2 * t + 1) ^ (t & 1);
  const Layout L(HD, P.block);
  const int pg = warp * (16 * kTiles) / P.block;   // page of the stage that holds the warp's keys
  const int k_in = warp * (16 * kTiles) - pg * P.block;   // first of them inside the page
  uint32_t qh[NT][KS][2], ql[kExact ? NT : 1][kExact ? KS : 1][2];
  float o[NT][KS][4], mref[NT][2], l[NT][2], cs[NT][2];
  int see[NT][2], all_seen = 0;
  bool fresh = true;
  int units = 0;
  for (int it = 0; it < len; ++it) {
    const int st = it % S::kStages;
    const Meta& m = sm.unit[units & 1];
    if (fresh) {                                   // Q comes while the first pages are on their way
      if (!warp_wait(&sm.unit_full[units & 1], (units >> 1) & 1, abort_flag, P.status)) return;
      fresh = false;
      const int mc = m.mc, m0 = m.m0, h = m.h, cu = m.cu, start = m.start, n = m.n;
      const float base = P.scale_log2 * (P.c.k_scale ? __ldg(P.c.k_scale + h) : 1.f);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int rr = j * 8 + g;                  // this lane's Q row
        float v[HD / 4];
#pragma unroll
        for (int i = 0; i < HD / 4; ++i) v[i] = 0.f;
        if (rr < mc) {
          const int i = (m0 + rr) / P.G, gg = (m0 + rr) - i * P.G;
          const T* src = static_cast<const T*>(P.q) + static_cast<long long>(cu + i) * P.q_stride +
                         (static_cast<long long>(h) * P.G + gg) * HD + t * (HD / 4);
          constexpr int E = 16 / sizeof(T);
#pragma unroll
          for (int k = 0; k < HD / 4 / E; ++k) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(src) + k);
            const T* p = reinterpret_cast<const T*>(&w);
#pragma unroll
            for (int y = 0; y < E; ++y) v[k * E + y] = to_f(p[y]);
          }
        }
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < HD / 4; ++i) mx = fmaxf(mx, fabsf(v[i]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // exponent that brings mx into [2^13, 2^14), in two factors so that neither overflows
        int ex = 0;
        if (mx > 0.f && mx <= FLT_MAX) ex = min(13 - ilogbf(mx), 126);
        const float f1 = exp2f(static_cast<float>(ex / 2)), f2 = exp2f(static_cast<float>(ex - ex / 2));
#pragma unroll
        for (int i = 0; i < KS; ++i) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float a = v[4 * i + 2 * y] * f1 * f2, c = v[4 * i + 2 * y + 1] * f1 * f2;
            qh[j][i][y] = pack2(a, c);
            if constexpr (kExact) {
              const float2 r = unpack2(qh[j][i][y]);
              ql[j][i][y] = pack2(a - r.x, c - r.y);
            }
          }
        }
        // the columns of S^T that this lane holds: rows 2t and 2t+1 of the tile
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int col = 2 * t + y, c_row = j * 8 + col;
          const int e = __shfl_sync(0xffffffffu, ex, col * 4);
          // never 0: a masked key's -inf times it has to stay -inf
          cs[j][y] = fmaxf(base * exp2f(static_cast<float>(-(e / 2))) * exp2f(static_cast<float>(-(e - e / 2))), FLT_MIN);
          const int pos = start + (m0 + c_row) / P.G;
          see[j][y] = c_row < mc ? (P.causal ? min(max(pos + 1, 0), n) : n) : 0;
          mref[j][y] = kFloor;
          l[j][y] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int y = 0; y < 4; ++y) o[j][i][y] = 0.f;
      }
      all_seen = m.seen;
    }
    if (!warp_wait(&sm.full[st], (it / S::kStages) & 1, abort_flag, P.status)) return;
    const int4 now = sm.step[st];
    const int key0 = pg == 0 ? now.x : now.y;
    const int kbase = key0 + k_in;                 // the warp's first key of the sequence
    if (key0 >= 0 && kbase < all_seen) {           // warp-uniform
      const uint8_t* rp = sm.ring[st] + pg * L.rec;
      // ---- S^T
      float s[kTiles][NT][4];
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        uint32_t kw[2][KW], ksc[2][2];             // K words and scales of two keys
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int key = k_in + 16 * u + gk + 8 * y;
          const uint8_t* p = rp + key * (HD / 2) + t * (HD / 8);
          if constexpr (HD == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            kw[y][0] = w.x; kw[y][1] = w.y; kw[y][2] = w.z; kw[y][3] = w.w;
            const uint32_t sc = e4m3x2(*reinterpret_cast<const uint16_t*>(rp + L.kscale() + key * 8 + 2 * t));
            ksc[y][0] = __byte_perm(sc, 0, 0x1010);
            ksc[y][1] = __byte_perm(sc, 0, 0x3232);
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(p);
            kw[y][0] = w.x; kw[y][1] = w.y;
            const uint32_t sc = rp[L.kscale() + key * 4 + t];
            ksc[y][0] = ksc[y][1] = e4m3x2(sc | (sc << 8));
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) s[u][j][0] = s[u][j][1] = s[u][j][2] = s[u][j][3] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t x[2][4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            e2m1x8_to_half2(kw[y][w], x[y]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[y][i] = mul2(x[y][i], ksc[y][HD == 128 ? w / 2 : 0]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a[4] = {x[0][2 * i], x[1][2 * i], x[0][2 * i + 1], x[1][2 * i + 1]};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma_f16(s[u][j], a, qh[j][2 * w + i][0], qh[j][2 * w + i][1]);
              if constexpr (kExact) mma_f16(s[u][j], a, ql[j][2 * w + i][0], ql[j][2 * w + i][1]);
            }
          }
        }
      }
      // ---- softmax: base-2 logits of keys gk, gk + 8 of each tile for rows 2t, 2t + 1
      constexpr int kSpan = 16 * kTiles;
      uint32_t ph[kTiles][NT][2], pl[kExact ? kTiles : 1][NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (kbase + kSpan > min(see[j][0], see[j][1])) {   // some key is behind a row's last
#pragma unroll
          for (int u = 0; u < kTiles; ++u)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (kbase + 16 * u + gk + 8 * (y >> 1) >= see[j][y & 1]) s[u][j][y] = -INFINITY;
        }
        float x[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float mx = fmaxf(s[0][j][y], s[0][j][2 + y]);
#pragma unroll
          for (int u = 1; u < kTiles; ++u) mx = fmax3(mx, s[u][j][y], s[u][j][2 + y]);
          x[y] = mx * cs[j][y];
        }
        // The max only has to be near: raised, for all keys of the warp, when it is
        // exceeded by 2^8.
        const bool raise = x[0] > mref[j][0] + (kHead + kRaise) || x[1] > mref[j][1] + (kHead + kRaise);
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], d));
            x[1] = fmaxf(x[1], __shfl_xor_sync(0xffffffffu, x[1], d));
          }
          float f[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float nm = fmaxf(mref[j][y], x[y] - kHead);
            f[y] = ex2_approx(mref[j][y] - nm);
            mref[j][y] = nm;
            l[j][y] *= f[y];
          }
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            o[j][i][0] *= f[0];
            o[j][i][1] *= f[1];
            o[j][i][2] *= f[0];
            o[j][i][3] *= f[1];
          }
        }
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
          float p[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) p[y] = ex2_approx(fmaf(s[u][j][y], cs[j][y & 1], -mref[j][y & 1]));
          l[j][0] += p[0] + p[2];
          l[j][1] += p[1] + p[3];
          const uint32_t h0 = pack2(p[0], p[1]), h1 = pack2(p[2], p[3]);
          ph[u][j][0] = transpose8x8(h0);
          ph[u][j][1] = transpose8x8(h1);
          if constexpr (kExact) {
            const float2 r0 = unpack2(h0), r1 = unpack2(h1);
            pl[u][j][0] = transpose8x8(pack2(p[0] - r0.x, p[1] - r0.y));
            pl[u][j][1] = transpose8x8(pack2(p[2] - r1.x, p[3] - r1.y));
          }
        }
      }
      // ---- O^T: V words of keys ka, kb and ka + 8, kb + 8 of each tile, and their scales
      constexpr int VW = HD / 64;                  // 32-bit words of a lane's HD/8 channels
      const bool edge = kbase + kSpan > all_seen;
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        uint32_t vw[4][VW], b[4], vsc[2];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int key = k_in + 16 * u + ((y & 1) ? kb : ka) + 8 * (y >> 1);
          const uint8_t* p = rp + L.vcodes() + key * (HD / 2) + g * (HD / 16);
          if constexpr (HD == 128) {
            const uint2 w = *reinterpret_cast<const uint2*>(p);
            vw[y][0] = w.x; vw[y][1] = w.y;
            b[y] = rp[L.vscale() + key * 8 + g];
          } else {
            vw[y][0] = *reinterpret_cast<const uint32_t*>(p);
            b[y] = rp[L.vscale() + key * 4 + (g >> 1)];
          }
        }
        if (edge) {
          // behind the last key that a row sees the page holds anything, NaN scales too
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (kbase + 16 * u + ((y & 1) ? kb : ka) + 8 * (y >> 1) >= all_seen) b[y] = 0;
        }
        vsc[0] = e4m3x2(b[0] | (b[1] << 8));
        vsc[1] = e4m3x2(b[2] | (b[3] << 8));
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          // two keys' codes of one channel side by side: the even channels, the odd ones
          uint32_t x[4][4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t c0 = vw[2 * y][w], c1 = vw[2 * y + 1][w];
            e2m1x8_to_half2((c0 & 0x0F0F0F0Fu) | ((c1 << 4) & 0xF0F0F0F0u), x[2 * y]);
            e2m1x8_to_half2(((c0 >> 4) & 0x0F0F0F0Fu) | (c1 & 0xF0F0F0F0u), x[2 * y + 1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a[4] = {mul2(x[0][i], vsc[0]), mul2(x[1][i], vsc[0]), mul2(x[2][i], vsc[1]),
                                   mul2(x[3][i], vsc[1])};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              if constexpr (kExact) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(d, a, pl[u][j][0], pl[u][j][1]);
                mma_f16(d, a, ph[u][j][0], ph[u][j][1]);
#pragma unroll
                for (int y = 0; y < 4; ++y) o[j][4 * w + i][y] += d[y];
              } else {
                mma_f16(o[j][4 * w + i], a, ph[u][j][0], ph[u][j][1]);
              }
            }
          }
        }
      }
    }
    if (!now.w) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[st]);
      continue;
    }
    // ------------------------------------------------------------ end of the unit's piece
    const int mc = m.mc, m0 = m.m0, h = m.h, cu = m.cu, begin = m.begin, end = m.end;
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sm.empty[st]);
      mbar_arrive(&sm.unit_empty[units & 1]);
    }
    fresh = true;
    const int par = units++ & 1;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[j][y] += __shfl_xor_sync(0xffffffffu, l[j][y], d);
        if (g == 0) {
          sm.mx[par][warp][j * 8 + 2 * t + y] = mref[j][y];
          sm.sum[par][warp][j * 8 + 2 * t + y] = l[j][y];
        }
      }
    if (!meet()) return;
    float f[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float mx = kFloor;
        for (int w = 0; w < kConsumers; ++w) mx = fmaxf(mx, sm.mx[par][w][j * 8 + 2 * t + y]);
        f[j][y] = ex2_approx(mref[j][y] - mx);
      }
    // lane's channels (HD/8) g + 2 i, + 1 of rows 2t, 2t + 1
    auto each = [&](auto&& fn) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            fn(j * 8 + 2 * t + y, g * (HD / 8) + 2 * i, o[j][i][y], o[j][i][2 + y], f[j][y]);
    };
    // Shared memory holds row 2t + y as row 4y + t and turns a lane group's HD/8 channels by
    // 2g: the stores of a warp then go to different banks.
    auto row_at = [](int row) { return (row & ~7) | ((row & 1) << 2) | ((row >> 1) & 3); };
    auto ch_at = [](int ch) {
      constexpr int W = HD / 8;
      return (ch & ~(W - 1)) | ((ch + 2 * (ch / W)) & (W - 1));
    };
    each([&](int row, int ch, float a, float b, float fac) {
      *reinterpret_cast<float2*>(&sm.slab[warp][row_at(row)][ch_at(ch)]) = make_float2(a * fac, b * fac);
    });
    if (!meet()) return;
    const bool whole = begin == end;
    float* mine = P.part + (static_cast<size_t>(blockIdx.x) * 2 + (begin == static_cast<int>(blockIdx.x) ? 1 : 0)) * S::kPart;
    const float vs = P.c.v_scale ? __ldg(P.c.v_scale + h) : 1.f;
    constexpr int kPer = RT * HD / 4 / (kConsumers * 32);   // float4 a thread
    static_assert(RT * HD / 4 % (kConsumers * 32) == 0, "");
    auto finish = [&](int row, int ch, float4 v, float mx, float sum) {
      if (row >= mc) return;
      const int i = (m0 + row) / P.G, gg = (m0 + row) - i * P.G;
      const size_t at = (static_cast<size_t>(cu + i) * P.c.H * P.G + static_cast<size_t>(h) * P.G + gg);
      const float inv = sum > 0.f || sum != sum ? vs / sum : 0.f;
      T* dst = static_cast<T*>(P.out) + at * HD + ch;
      if constexpr (kExact) {
        *reinterpret_cast<float4*>(dst) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
      } else {
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
      }
      if (P.lse && ch == 0) P.lse[at] = sum > 0.f || sum != sum ? (mx + log2f(sum)) * kLn2 : -INFINITY;
    };
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int at = (threadIdx.x + k * kConsumers * 32) * 4;
      const int row = at / HD, ch = at % HD;
      float mx = kFloor;
      for (int w = 0; w < kConsumers; ++w) mx = fmaxf(mx, sm.mx[par][w][row]);
      float sum = 0.f;
      for (int w = 0; w < kConsumers; ++w) sum += sm.sum[par][w][row] * ex2_approx(sm.mx[par][w][row] - mx);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) {
        const float2 a = *reinterpret_cast<const float2*>(&sm.slab[w][row_at(row)][ch_at(ch)]);
        const float2 c = *reinterpret_cast<const float2*>(&sm.slab[w][row_at(row)][ch_at(ch + 2)]);
        v.x += a.x; v.y += a.y; v.z += c.x; v.w += c.y;
      }
      if (whole) {
        finish(row, ch, v, mx, sum);
      } else {
        *reinterpret_cast<float4*>(mine + row * HD + ch) = v;
        if (ch == 0) {
          mine[RT * HD + row] = mx;
          mine[RT * HD + RT + row] = sum;
        }
      }
    }
    if (whole) continue;
    // ---- the unit lies in blocks begin .. end: who finds all parts there joins them in order
    // (one warp's fences, between the barriers, cover the whole block's stores and loads)
    if (!meet()) return;
    if (warp == 0) {
      const bool all = leave_part(P.left, P.status.call, begin, end, [&](int i) { return 2 * i + (i == begin ? 1 : 0); });
      if (lane == 0) sm.joiner = all;
    }
    if (!meet()) return;
    if (!sm.joiner) continue;
    auto part_of = [&](int i) {
      return P.part + (static_cast<size_t>(i) * 2 + (i == begin ? 1 : 0)) * S::kPart;
    };
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int at = (threadIdx.x + k * kConsumers * 32) * 4;
      const int row = at / HD, ch = at % HD;
      if (row >= mc) continue;
      // eight parts' loads at a time; the running maximum and sums as in a softmax
      float mx = kFloor, sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int kBatch = 8;
      for (int i0 = begin; i0 <= end; i0 += kBatch) {
        float pm[kBatch], ps[kBatch];
        float4 pv[kBatch];
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
          const float* p = part_of(min(i0 + y, end));
          pm[y] = __ldcg(p + RT * HD + row);
          ps[y] = __ldcg(p + RT * HD + RT + row);
          pv[y] = __ldcg(reinterpret_cast<const float4*>(p + row * HD + ch));
        }
        float top = mx;
#pragma unroll
        for (int y = 0; y < kBatch; ++y) top = fmaxf(top, pm[y]);
        const float old = ex2_approx(mx - top);
        sum *= old;
        v.x *= old; v.y *= old; v.z *= old; v.w *= old;
        mx = top;
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
          const float fac = i0 + y <= end ? ex2_approx(pm[y] - mx) : 0.f;
          sum = fmaf(ps[y], fac, sum);
          v.x = fmaf(pv[y].x, fac, v.x); v.y = fmaf(pv[y].y, fac, v.y);
          v.z = fmaf(pv[y].z, fac, v.z); v.w = fmaf(pv[y].w, fac, v.w);
        }
      }
      finish(row, ch, v, mx, sum);
    }
  }
}

// Workspace behind the header: flags of the parts left, then the partial results.
constexpr int kMaxBlocks = 448;                    // three blocks on each of 148 SMs
constexpr int kMaxChunkBlocks = 160;
static_assert(kMaxChunkBlocks * 4 <= kMaxBlocks * 2, "");

size_t chunk_part_bytes(int d, int grid);
cudaError_t launch_chunk(const AttnParams& P, int d, int grid, cudaStream_t st);

// Where the 128-row tiles of kv4_chunk.cu take over (the fp32 path and lists stay here). Measured
// at d 128 in us, with units of sixteen rows here / there:
//   16 sequences of 8k to 16k, 8 KV heads: 9 rows 125/246, 20 rows 181/247, 32 rows 231/248, 40 rows 280/248
//   one sequence of 32k, 12 KV heads: 9 rows 51/83, 20 rows 66/83, 32 rows 70/84, 40 rows 95/84
static bool many_rows(int max_q, int G) { return static_cast<long long>(max_q) * G > 32; }

// Bytes of the flags, two a block (here) or four (kMaxChunkBlocks); cleared before a captured call.
size_t attn_ws_clear() { return align_up(kMaxBlocks * 2 * sizeof(unsigned long long), 256); }
size_t attn_ws_bytes(int d, int max_q, int G) {
  const size_t few = static_cast<size_t>(kMaxBlocks) * 2 * (16 * d + 32) * sizeof(float);
  const size_t part = many_rows(max_q, G) ? max(few, chunk_part_bytes(d, kMaxChunkBlocks)) : few;
  return attn_ws_clear() + part;
}

template <typename T, int HD, int NT>
static cudaError_t launch_stream(const AttnParams& P, int num_sms, cudaStream_t st) {
  const int smem = static_cast<int>(sizeof(AttnSmem<HD, NT>));
  cudaError_t e = cudaFuncSetAttribute(attn_stream_kernel<T, HD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = min(kMaxBlocks, num_sms * (NT == 1 ? 3 : 2));
  attn_stream_kernel<T, HD, NT><<<grid, kThreads, smem, st>>>(P);
  return cudaGetLastError();
}

cudaError_t launch_attn(const Cache& c, const Batch& bt, const void* q, long long q_stride, int Hq, void* out,
                        float* lse, bool bf16, float scale, int causal, int d, int block, int max_q, const int* kv_idx,
                        const int* kv_cnt, const Status& status, uint8_t* ws, int num_sms, cudaStream_t st) {
  AttnParams P;
  P.c = c;
  P.bt = bt;
  P.q = q;
  P.q_stride = q_stride;
  P.out = out;
  P.lse = lse;
  P.kv_idx = kv_idx;
  P.kv_cnt = kv_cnt;
  P.scale_log2 = scale * 1.4426950408889634f;
  P.G = Hq / c.H;
  P.causal = causal;
  P.block = block;
  P.status = status;
  P.left = reinterpret_cast<unsigned long long*>(ws);
  P.part = reinterpret_cast<float*>(ws + attn_ws_clear());
  if (bf16 && !kv_idx && many_rows(max_q, P.G)) return launch_chunk(P, d, min(kMaxChunkBlocks, num_sms), st);
  // Up to eight query rows a unit, or sixteen. The calls measured above do not bear this border out:
  // with units of eight they take 73, 128, 176, 209 and 38, 48, 61, 71 us.
  const bool few = (kv_idx ? P.G : static_cast<long long>(max_q) * P.G) <= 8;
#define FVATTN_KV4(T, HD) (few ? launch_stream<T, HD, 1>(P, num_sms, st) : launch_stream<T, HD, 2>(P, num_sms, st))
  if (bf16) return d == 128 ? FVATTN_KV4(__nv_bfloat16, 128) : FVATTN_KV4(__nv_bfloat16, 64);
  return d == 128 ? FVATTN_KV4(float, 128) : FVATTN_KV4(float, 64);
#undef FVATTN_KV4
}

}  // namespace kv4
}  // namespace fvattn
