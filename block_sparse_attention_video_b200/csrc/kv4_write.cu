// kv4_write.cu -- the 4-bit cache's writing and reading back: K and V rows to E2M1
// codes with one E4M3 scale per 16 channels, exact page sums of the keys, and rows
// of the cache to bf16 or fp32.
//
// Quantization of 16 channels x: s = E4M3 nearest to min(max|x| / 6, 448), code =
// E2M1 nearest to x / s, ties to even. The codes are exact decisions: r = 1/s to 2^-22, q0 =
// fl(x r), q = fl(q0 + r (x - q0 s)); the residual x - q0 s is exact (fma), so q is x / s up to
// 2^-44 before its last rounding. Where x / s lies on a border t of two codes (t s has at most
// 7 significant bits), q = t exactly. Where it does not, x is at least one fp32 step away from
// t s, and because s < 2 (as a significand) that is more than 1/1.875 = 0.53 steps of t, so q
// does not round onto t. The same holds for max|x| / 6 and the borders of E4M3.
//
// Both kernels move bytes: what bounds them is HBM (2 d es bytes of K and V a token
// and head, d + d/8 bytes of codes and scales).
#include "kv4_units.cuh"
#include "sm100.cuh"

namespace fvattn {
namespace kv4 {

constexpr int kWriteThreads = 256;

// Eight elements as they lie in memory, and as fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// x / y for one y and many x: r = fl(1/y), q0 = fl(x r), then Markstein's correction
// ("Computation of elementary functions on the IBM RISC System/6000", 1990) with the exact
// residual of a fused multiply-add, twice: the first makes q faithful, the second correctly
// rounded. For y in [2^-60, 2^60] and |x| <= most = 2^13 y, where larger ones saturate anyway.
struct Divisor {
  float y, r, most;
  int kind;               // 0: y is 1 (no scale), 1: corrected product, 2: plain division
  __device__ Divisor(const float* scales, int h) {
    y = scales ? __ldg(scales + h) : 1.f;
    r = 1.f / y;
    kind = !scales ? 0 : y >= 0x1p-60f && y <= 0x1p60f ? 1 : 2;
    most = 8192.f * y;    // infinite for huge y: then nothing is clamped
  }
  __device__ __forceinline__ float corrected(float x) const {
    float q = x * r;
    q = fmaf(fmaf(-q, y, x), r, q);
    return fmaf(fmaf(-q, y, x), r, q);
  }
};

// Two products, and two quotients corrected once: q + r (x - q y) of q = x r. The packed
// operations take one issue slot for two values; issue slots are what bounds the kernel next.
__device__ __forceinline__ float2 corrected2(float2 x, float2 q, float2 minus_y, float2 r) {
  return __ffma2_rn(__ffma2_rn(q, minus_y, x), r, q);
}

__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Eight channels of a row, the other half of the 16-channel group in the neighbouring
// lane: codes (lowest channel in the low bits) and the group's scale code. Whole warp.
// The quotients m / 6 and x / s are corrected once: they are then x / s up to 2^-44 before
// the last rounding, which is all that the borders need (above).
template <typename T>
__device__ __forceinline__ uint32_t quantize8(const Raw8<T>& raw, const Divisor& head, uint32_t& scale) {
  float x[8];
  raw.get(x);
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 7; i += 2) m = fmax3(m, fabsf(x[i]), fabsf(x[i + 1]));
  m = fmaxf(m, fabsf(x[7]));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if (m > head.most) {    // infinities, and what saturates by far
    m = head.most;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -head.most), head.most);
  }
  if (head.kind == 1) {   // division is monotonic: the largest quotient is the largest's
    m = head.corrected(m);
    const float2 r2 = make_float2(head.r, head.r), y2 = make_float2(-head.y, -head.y);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 v = make_float2(x[i], x[i + 1]);
      float2 q = __fmul2_rn(v, r2);
      q = corrected2(v, q, y2, r2);
      q = corrected2(v, q, y2, r2);
      x[i] = q.x;
      x[i + 1] = q.y;
    }
  } else if (head.kind == 2) {
    m = m / head.y;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i] / head.y, -8192.f), 8192.f);
  }
  float c = m * 0.166666672f;                 // fl(1/6)
  c = fmaf(fmaf(-c, 6.f, m), 0.166666672f, c);
  scale = float_to_e4m3(fminf(c, 448.f));     // 448 where an infinite m has made c a NaN
  const float s = e4m3_to_float(scale);
  // Codes of zero where the scale is. (Some come out as minus zero; to make them plus costs 2% of the
  // kernel: 9,360 tokens x 40 scaled heads 76.3 to 78.2 us.)
  const float r = scale == 0u ? 0.f : reciprocal(s);
  const float2 r2 = make_float2(r, r), s2 = make_float2(-s, -s);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 v = make_float2(x[i], x[i + 1]);
    const float2 d = corrected2(v, __fmul2_rn(v, r2), s2, r2);
    q[i] = d.x;
    q[i + 1] = d.y;
  }
  return pack_e2m1x8(q);
}

// Adds eight stored values, in units of 2^-10, to integer sums. A value is a whole number
// below 2^22 of them: added to 1.5 * 2^23 it stands in the low bits of the sum, whose own bits
// (kMagic, once per call) are taken off at the end.
constexpr uint32_t kMagic = 0x4B400000u;
__device__ __forceinline__ void add8(uint32_t codes, uint32_t scale, uint32_t (&acc)[8]) {
  uint32_t p[4];
  e2m1x8_to_half2(codes, p);
  const float s = e4m3_to_float(scale) * 1024.f;
  const float2 s2 = make_float2(s, s), magic = make_float2(12582912.f, 12582912.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __ffma2_rn(__half22float2(*reinterpret_cast<const __half2*>(&p[i])), s2, magic);
    acc[2 * i] += __float_as_uint(f.x);
    acc[2 * i + 1] += __float_as_uint(f.y);
  }
}

// One block per (page of a sequence that the call's rows touch, KV head): quantizes the
// rows that fall into the page, HD/8 lanes a row, and if the page is full then, adds up
// its keys (the codes just made, and the older ones from the page). Pages are enumerated
// without a prefix sum: sequence b owns the tiles from cu[b]/block + 2b on, which leaves room
// for the at most q/block + 2 pages that q rows touch. The sum is one of integers: exact and
// the same in any order.
template <typename T, int HD>
__global__ void __launch_bounds__(kWriteThreads, sizeof(T) == 2 ? 4 : 3)
    append_kernel(const Cache c, const Batch bt, const T* __restrict__ k, const T* __restrict__ v,
                  long long k_stride, long long v_stride, int block, const Status status) {
  constexpr int LPR = HD / 8;                 // lanes per row
  constexpr int RPB = kWriteThreads / LPR;    // rows per pass of the block
  __shared__ Seqs seqs;
  open_call(status);
  seqs.load<kWriteThreads>(bt);
  __syncthreads();
  const int *cu = seqs.rows_of(bt), *kv_len = seqs.lengths_of(bt);
  const int h = blockIdx.x % c.H;
  const int tile = blockIdx.x / c.H;
  check_rows(bt, cu, status);
  int lo = 0, hi = bt.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] / block + 2 * mid <= tile) lo = mid; else hi = mid;
  }
  const int b = lo;
  const int r0 = cu[b];
  const int q = cu[b + 1] - r0;
  if (q <= 0 || r0 < 0) return;
  const int n = held(kv_len[b], bt, block, status);
  const int start = start_of(kv_len[b], q);   // position of row r0
  if (start < 0 && threadIdx.x == 0) record_status(status, FVATTN_ERR_INVALID_ARG);
  if (start >= n) return;                     // all behind the table's end (recorded above)
  const int nth = tile - (r0 / block + 2 * b);   // of the pages that the rows touch
  if (nth < 0) return;                        // a tile of the rows before cu[0]
  const int pg = max(start, 0) / block + nth;
  const int first = max(start, pg * block);   // positions [first, last) of this block
  const int last = min(min(n, (pg + 1) * block), start + rows_end(bt, cu) - r0);
  if (first >= last) return;
  const int slot = pool_slot(bt, c.num_pages, b, pg, status);
  if (slot < 0) return;
  const Layout L(HD, block);
  uint8_t* rec = c.pages + (static_cast<size_t>(slot) * c.H + h) * L.rec;
  const Divisor ks(c.k_scale, h), vs(c.v_scale, h);
  const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
  const bool full = c.ksum && last == (pg + 1) * block;      // block-uniform
  uint32_t acc[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  uint32_t added = 0u;
  const T* kp = k + static_cast<long long>(r0 - start) * k_stride + h * HD + l * 8;   // of position 0
  const T* vp = v + static_cast<long long>(r0 - start) * v_stride + h * HD + l * 8;
  // 0, but not to the compiler: CUDA 12.9 passes a word of codes from the conversion that packs it
  // on to the one that unpacks it without its upper half.
  const uint32_t zero = static_cast<uint32_t>(block) >> 16;
  Raw8<T> x, y, xn, yn;                       // a row's K and V, the next one's while it is quantized
  int pos = first + g;
  x.load(kp + static_cast<long long>(min(pos, last - 1)) * k_stride);
  y.load(vp + static_cast<long long>(min(pos, last - 1)) * v_stride);
  // a warp's rows go round together: lanes without one repeat the last row and store nothing
  const int warp_first = first + (threadIdx.x & ~31) / LPR;
  for (int base = warp_first; base < last; base += RPB, pos += RPB) {
    const int t = pos - pg * block;
    const bool mine = pos < last;
    if (base + RPB < last) {
      const int next = min(pos + RPB, last - 1);
      xn.load(kp + static_cast<long long>(next) * k_stride);
      yn.load(vp + static_cast<long long>(next) * v_stride);
    }
    uint32_t sc;
    uint32_t w = quantize8(x, ks, sc);
    if (mine) {
      *reinterpret_cast<uint32_t*>(rec + t * (HD / 2) + l * 4) = w;
      if (!(l & 1)) rec[L.kscale() + t * (HD / kGroup) + (l >> 1)] = static_cast<uint8_t>(sc);
      if (full) {
        add8(w | zero, sc, acc);
        ++added;
      }
    }
    w = quantize8(y, vs, sc);
    if (mine) {
      *reinterpret_cast<uint32_t*>(rec + L.vcodes() + t * (HD / 2) + l * 4) = w;
      if (!(l & 1)) rec[L.vscale() + t * (HD / kGroup) + (l >> 1)] = static_cast<uint8_t>(sc);
    }
    x = xn;
    y = yn;
  }
  if (!full) return;
  for (int t = g; t < first - pg * block; t += RPB, ++added)
    add8(*reinterpret_cast<const uint32_t*>(rec + t * (HD / 2) + l * 4),
         rec[L.kscale() + t * (HD / kGroup) + (l >> 1)], acc);
  __shared__ uint32_t part[RPB][HD];
#pragma unroll
  for (int i = 0; i < 8; ++i) part[g][l * 8 + i] = acc[i] - added * kMagic;
  __syncthreads();
  if (threadIdx.x < HD) {
    uint32_t s = 0u;
#pragma unroll 8
    for (int i = 0; i < RPB; ++i) s += part[i][threadIdx.x];
    c.ksum[(static_cast<size_t>(slot) * c.H + h) * HD + threadIdx.x] = static_cast<int>(s);
  }
}

// Eight codes to T. A code times its scale is exact in fp16; the head's scale, where there is one,
// is the one fp32 rounding.
template <typename T>
__device__ __forceinline__ void decode8(uint32_t codes, uint32_t scale, const float* head_scales, int h, T* out) {
  const __half2 two = e4m3x2_to_half2(scale | scale << 8);
  const float hs = head_scales ? __ldg(head_scales + h) : 1.f;
  uint32_t p[4];
  e2m1x8_to_half2(codes, p);
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&p[i]), two));
    if (head_scales) f = __fmul2_rn(f, make_float2(hs, hs));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  store8(out, x);
}

// A block reads EACH (row, KV head) pairs for every group of HD/8 lanes, neighbouring groups on
// neighbouring heads so that the outputs are written in one stream. Where the block's rows
// lie is looked up once, a thread a row.
template <typename T, int HD, int EACH>
__global__ void __launch_bounds__(kWriteThreads)
    read_kernel(const Cache c, const Batch bt, T* __restrict__ k_out, T* __restrict__ v_out, int block, const Status status) {
  constexpr int LPR = HD / 8, GROUPS = kWriteThreads / LPR, UNITS = GROUPS * EACH;
  constexpr int BATCH = EACH < 4 ? EACH : 4;          // pairs whose loads are in flight together
  __shared__ int2 place[UNITS + 1];                   // pool slot (-1: invalid, -2: no row) and position in the page
  __shared__ Seqs seqs;
  open_call(status);
  seqs.load<kWriteThreads>(bt);
  __syncthreads();
  const int *cu = seqs.rows_of(bt), *kv_len = seqs.lengths_of(bt);
  check_rows(bt, cu, status);
  const unsigned H = static_cast<unsigned>(c.H), u0 = blockIdx.x * UNITS;
  const unsigned row0 = u0 / H, rows = min(u0 + UNITS - 1, bt.rows * H - 1) / H - row0 + 1;
  for (unsigned i = threadIdx.x; i < rows; i += kWriteThreads) {
    const int r = static_cast<int>(row0 + i);
    int slot = -2, t = 0;
    if (r < cu[bt.B]) {
      int lo = 0, hi = bt.B;                          // cu[lo] <= r < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= r) lo = mid; else hi = mid;
      }
      const int b = lo;
      if (cu[b] >= 0 && r >= cu[b]) {
        const int n = held(kv_len[b], bt, block, status), pos = start_of(kv_len[b], cu[b + 1] - r);
        slot = -1;
        if (pos >= 0 && pos < n) slot = pool_slot(bt, c.num_pages, b, pos / block, status);
        else record_status(status, FVATTN_ERR_INVALID_ARG);
        t = pos >= 0 ? pos % block : 0;
      }
    }
    place[i] = make_int2(slot, t);
  }
  __syncthreads();
  const Layout L(HD, block);
  const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
#pragma unroll
  for (int part = 0; part < EACH; part += BATCH) {
    uint32_t w[BATCH][2], sc[BATCH][2];
    int slot[BATCH];
    unsigned head[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const unsigned u = u0 + (part + i) * GROUPS + g, r = u / H;
      slot[i] = -2;
      head[i] = u - r * H;
      if (u < bt.rows * H) {
        const int2 at = place[r - row0];
        slot[i] = at.x;
        if (at.x >= 0) {
          const uint8_t* rec = c.pages + (static_cast<size_t>(at.x) * H + head[i]) * L.rec;
          const int co = at.y * (HD / 2) + l * 4, so = at.y * (HD / kGroup) + (l >> 1);
          w[i][0] = __ldg(reinterpret_cast<const uint32_t*>(rec + co));
          sc[i][0] = __ldg(rec + L.kscale() + so);
          w[i][1] = __ldg(reinterpret_cast<const uint32_t*>(rec + L.vcodes() + co));
          sc[i][1] = __ldg(rec + L.vscale() + so);
        } else {
          w[i][0] = w[i][1] = sc[i][0] = sc[i][1] = 0u;   // zeros
        }
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (slot[i] == -2) continue;
      const size_t at = static_cast<size_t>(u0 + (part + i) * GROUPS + g) * HD + l * 8;
      decode8(w[i][0], sc[i][0], c.k_scale, head[i], k_out + at);
      decode8(w[i][1], sc[i][1], c.v_scale, head[i], v_out + at);
    }
  }
}

template <typename T>
static cudaError_t append_t(const Cache& c, const Batch& bt, const void* k, const void* v, long long ks,
                            long long vs, int d, int block, const Status& status, cudaStream_t st) {
  const long long grid = (static_cast<long long>(bt.rows) / block + 2ll * bt.B) * c.H;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const T* kt = static_cast<const T*>(k);
  const T* vt = static_cast<const T*>(v);
  if (d == 128)
    append_kernel<T, 128><<<static_cast<unsigned>(grid), kWriteThreads, 0, st>>>(c, bt, kt, vt, ks, vs, block, status);
  else
    append_kernel<T, 64><<<static_cast<unsigned>(grid), kWriteThreads, 0, st>>>(c, bt, kt, vt, ks, vs, block, status);
  return cudaGetLastError();
}

template <typename T, int HD, int EACH>
static cudaError_t read_launch(const Cache& c, const Batch& bt, void* k, void* v, int block, const Status& status,
                               cudaStream_t st) {
  const long long per = kWriteThreads / (HD / 8) * EACH;
  const long long grid = (static_cast<long long>(bt.rows) * c.H + per - 1) / per;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  read_kernel<T, HD, EACH><<<static_cast<unsigned>(grid), kWriteThreads, 0, st>>>(c, bt, static_cast<T*>(k),
                                                                                static_cast<T*>(v), block, status);
  return cudaGetLastError();
}

template <typename T, int HD>
static cudaError_t read_hd(const Cache& c, const Batch& bt, void* k, void* v, int block, const Status& status,
                           cudaStream_t st) {
  // Eight pairs a lane group share the block's look-ups (393,120 pairs at d 128: 53 us, 68 with
  // one); one where eight would leave SMs without a block (3,700 pairs at d 64: 4.2 us, 8.6 with
  // eight).
  if (static_cast<long long>(bt.rows) * c.H < 148ll * 8 * (kWriteThreads / (HD / 8)))
    return read_launch<T, HD, 1>(c, bt, k, v, block, status, st);
  return read_launch<T, HD, 8>(c, bt, k, v, block, status, st);
}

template <typename T>
static cudaError_t read_t(const Cache& c, const Batch& bt, void* k, void* v, int d, int block, const Status& status,
                          cudaStream_t st) {
  return d == 128 ? read_hd<T, 128>(c, bt, k, v, block, status, st) : read_hd<T, 64>(c, bt, k, v, block, status, st);
}

cudaError_t launch_append(const Cache& c, const Batch& bt, const void* k, const void* v, long long ks,
                          long long vs, bool bf16, int d, int block, const Status& status, cudaStream_t st) {
  return bf16 ? append_t<__nv_bfloat16>(c, bt, k, v, ks, vs, d, block, status, st)
              : append_t<float>(c, bt, k, v, ks, vs, d, block, status, st);
}

cudaError_t launch_read(const Cache& c, const Batch& bt, void* k, void* v, bool bf16, int d, int block,
                        const Status& status, cudaStream_t st) {
  return bf16 ? read_t<__nv_bfloat16>(c, bt, k, v, d, block, status, st)
              : read_t<float>(c, bt, k, v, d, block, status, st);
}

}  // namespace kv4
}  // namespace fvattn
