// kv4_write.cu -- the 4-bit cache's writing and reading back: K and V rows to E2M1
// codes with one E4M3 scale per 16 channels, exact page sums of the keys, and rows
// of the cache to bf16 or fp32.
//
// Quantization of 16 channels x: s = E4M3 nearest to min(max|x| / 6, 448), code =
// E2M1 nearest to x / s, ties to even. The codes are exact decisions: r = fl(1/s),
// q0 = fl(x r), q = fl(q0 + r fl(x - q0 s)); the residual x - q0 s is exact (fma), so
// q is x / s up to 2^-47 before its last rounding. Where x / s lies on a border t of
// two codes (t s has at most 7 significant bits), q = t exactly. Where it does not, x
// is at least one fp32 step away from t s, and because s < 2 (as a significand) that
// is more than 1/1.875 = 0.53 steps of t, so q does not round onto t.
//
// Both kernels move bytes: what bounds them is HBM (2 d es bytes of K and V a token
// and head, d + d/8 bytes of codes and scales).
#include "kv4.cuh"
#include "sm100.cuh"

namespace fvattn {
namespace kv4 {

constexpr int kWriteThreads = 256;

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Eight channels of a row, the other half of the 16-channel group in the neighbouring
// lane: codes (lowest channel in the low bits) and the group's scale code. `mask` names
// the lanes that call this together.
__device__ __forceinline__ uint32_t quantize8(float (&x)[8], float head_scale, unsigned mask, uint32_t& scale) {
  if (head_scale != 1.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], head_scale);
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  m = fmaxf(m, __shfl_xor_sync(mask, m, 1));
  scale = float_to_e4m3(fminf(__fdiv_rn(m, 6.f), 448.f));
  if (scale == 0u) return 0u;
  const float s = e4m3_to_float(scale);
  if (m > 4096.f) {   // keeps the residual finite; |x| >= 6 s is code 6 whatever it is
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -4096.f), 4096.f);
  }
  const float r = __fdiv_rn(1.f, s);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q0 = x[i] * r;
    q[i] = fmaf(fmaf(-q0, s, x[i]), r, q0);
  }
  return pack_e2m1x8(q);
}

// One block per (page of a sequence that the call's rows touch, KV head): quantizes the
// rows that fall into the page, HD/8 lanes a row, and if the page is full then, adds up
// its keys' codes (the older ones with them). Pages are enumerated without a prefix
// sum: sequence b owns the tiles from cu[b]/block + 2b on, which leaves room for the
// at most q/block + 2 pages that q rows touch. The sum is a sum of integers: exact and
// the same in any order.
template <typename T, int HD>
__global__ void __launch_bounds__(kWriteThreads)
    append_kernel(const Cache c, const Batch bt, const T* __restrict__ k, const T* __restrict__ v,
                  long long k_stride, long long v_stride, int block, int* status) {
  constexpr int LPR = HD / 8;                 // lanes per row
  constexpr int RPB = kWriteThreads / LPR;    // rows per pass of the block
  const int h = blockIdx.x % c.H;
  const int tile = blockIdx.x / c.H;
  if (blockIdx.x == 0 && threadIdx.x == 0 && __ldg(bt.cu + bt.B) > bt.rows)
    record_status(status, FVATTN_ERR_INVALID_ARG);
  int lo = 0, hi = bt.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(bt.cu + mid) / block + 2 * mid <= tile) lo = mid; else hi = mid;
  }
  const int b = lo;
  const int r0 = __ldg(bt.cu + b);
  const int q = __ldg(bt.cu + b + 1) - r0;
  if (q <= 0) return;
  const int n = held(bt, b, block, status);
  const int start = n - q;                    // position of row r0
  if (start < 0 && threadIdx.x == 0) record_status(status, FVATTN_ERR_INVALID_ARG);
  const int pg = max(start, 0) / block + tile - (r0 / block + 2 * b);
  const int first = max(start, pg * block);   // positions [first, last) of this block
  const int last = min(n, (pg + 1) * block);
  if (first >= last) return;
  const int slot = pool_slot(bt, c.num_pages, b, pg, status);
  if (slot < 0) return;
  const Layout L(HD, block);
  uint8_t* rec = c.pages + (static_cast<size_t>(slot) * c.H + h) * L.rec;
  const float ks = c.k_scale ? __ldg(c.k_scale + h) : 1.f;
  const float vs = c.v_scale ? __ldg(c.v_scale + h) : 1.f;
  const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
  const unsigned mask = 0x3u << ((threadIdx.x & 31) & ~1);   // the two lanes of a group
  for (int pos = first + g; pos < last; pos += RPB) {
    const int r = r0 + pos - start;
    if (r >= bt.rows) break;
    const int t = pos - pg * block;
    float x[8];
    uint32_t sc;
    load8(k + static_cast<long long>(r) * k_stride + h * HD + l * 8, x);
    uint32_t w = quantize8(x, ks, mask, sc);
    *reinterpret_cast<uint32_t*>(rec + t * (HD / 2) + l * 4) = w;
    if (!(l & 1)) rec[L.kscale() + t * (HD / kGroup) + (l >> 1)] = static_cast<uint8_t>(sc);
    load8(v + static_cast<long long>(r) * v_stride + h * HD + l * 8, x);
    w = quantize8(x, vs, mask, sc);
    *reinterpret_cast<uint32_t*>(rec + L.vcodes() + t * (HD / 2) + l * 4) = w;
    if (!(l & 1)) rec[L.vscale() + t * (HD / kGroup) + (l >> 1)] = static_cast<uint8_t>(sc);
  }
  if (!c.ksum || last != (pg + 1) * block) return;   // block-uniform
  // The page is full. Its codes are read back: this block's own stores are visible to
  // it after the barrier, the older ones came from earlier calls.
  __shared__ int part[RPB][HD];
  __syncthreads();
  int acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int t = g; t < block; t += RPB) {
    const uint32_t w = *reinterpret_cast<const volatile uint32_t*>(rec + t * (HD / 2) + l * 4);
    const uint32_t sc = *reinterpret_cast<const volatile uint8_t*>(rec + L.kscale() + t * (HD / kGroup) + (l >> 1));
    uint32_t p[4];
    e2m1x8_to_half2(w, p);
    const float s = e4m3_to_float(sc) * 1024.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
      acc[2 * i] += __float2int_rn(f.x * s);          // a whole number below 2^22: exact
      acc[2 * i + 1] += __float2int_rn(f.y * s);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[g][l * 8 + i] = acc[i];
  __syncthreads();
  if (threadIdx.x < HD) {
    int s = 0;
#pragma unroll 8
    for (int i = 0; i < RPB; ++i) s += part[i][threadIdx.x];
    c.ksum[(static_cast<size_t>(slot) * c.H + h) * HD + threadIdx.x] = s;
  }
}

template <typename T>
__device__ __forceinline__ void decode8(const uint8_t* codes, const uint8_t* scale, float head_scale, T* out) {
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes));
  const float s = e4m3_to_float(__ldg(scale));
  uint32_t p[4];
  e2m1x8_to_half2(w, p);
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
    x[2 * i] = f.x * s * head_scale;                  // f * s is exact: one rounding
    x[2 * i + 1] = f.y * s * head_scale;
  }
  store8(out, x);
}

// HD/8 lanes per (row, KV head), neighbouring groups on neighbouring heads of a row so
// that the outputs are written in one stream.
template <typename T, int HD>
__global__ void __launch_bounds__(kWriteThreads)
    read_kernel(const Cache c, const Batch bt, T* __restrict__ k_out, T* __restrict__ v_out, int block, int* status) {
  constexpr int LPR = HD / 8;
  const long long unit = static_cast<long long>(blockIdx.x) * (kWriteThreads / LPR) + threadIdx.x / LPR;
  const int l = threadIdx.x % LPR;
  if (blockIdx.x == 0 && threadIdx.x == 0 && __ldg(bt.cu + bt.B) > bt.rows)
    record_status(status, FVATTN_ERR_INVALID_ARG);
  const int r = static_cast<int>(unit / c.H);
  const int h = static_cast<int>(unit - static_cast<long long>(r) * c.H);
  if (r >= bt.rows) return;
  int b;
  if (!sequence_of(bt, r, b)) return;
  const int n = held(bt, b, block, status);
  const int pos = n - (__ldg(bt.cu + b + 1) - r);
  int slot = -1;
  if (pos >= 0 && pos < n) slot = pool_slot(bt, c.num_pages, b, pos / block, status);
  else record_status(status, FVATTN_ERR_INVALID_ARG);
  T* ko = k_out + static_cast<size_t>(unit) * HD + l * 8;
  T* vo = v_out + static_cast<size_t>(unit) * HD + l * 8;
  if (slot < 0) {
    const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    store8(ko, z);
    store8(vo, z);
    return;
  }
  const Layout L(HD, block);
  const uint8_t* rec = c.pages + (static_cast<size_t>(slot) * c.H + h) * L.rec;
  const int t = pos % block;
  decode8(rec + t * (HD / 2) + l * 4, rec + L.kscale() + t * (HD / kGroup) + (l >> 1),
          c.k_scale ? __ldg(c.k_scale + h) : 1.f, ko);
  decode8(rec + L.vcodes() + t * (HD / 2) + l * 4, rec + L.vscale() + t * (HD / kGroup) + (l >> 1),
          c.v_scale ? __ldg(c.v_scale + h) : 1.f, vo);
}

template <typename T>
static cudaError_t append_t(const Cache& c, const Batch& bt, const void* k, const void* v, long long ks,
                            long long vs, int d, int block, int* status, cudaStream_t st) {
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

template <typename T>
static cudaError_t read_t(const Cache& c, const Batch& bt, void* k, void* v, int d, int block, int* status,
                          cudaStream_t st) {
  const long long per = kWriteThreads / (d / 8);
  const long long grid = (static_cast<long long>(bt.rows) * c.H + per - 1) / per;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  T* kt = static_cast<T*>(k);
  T* vt = static_cast<T*>(v);
  if (d == 128)
    read_kernel<T, 128><<<static_cast<unsigned>(grid), kWriteThreads, 0, st>>>(c, bt, kt, vt, block, status);
  else
    read_kernel<T, 64><<<static_cast<unsigned>(grid), kWriteThreads, 0, st>>>(c, bt, kt, vt, block, status);
  return cudaGetLastError();
}

cudaError_t launch_append(const Cache& c, const Batch& bt, const void* k, const void* v, long long ks,
                          long long vs, bool bf16, int d, int block, int* status, cudaStream_t st) {
  return bf16 ? append_t<__nv_bfloat16>(c, bt, k, v, ks, vs, d, block, status, st)
              : append_t<float>(c, bt, k, v, ks, vs, d, block, status, st);
}

cudaError_t launch_read(const Cache& c, const Batch& bt, void* k, void* v, bool bf16, int d, int block,
                        int* status, cudaStream_t st) {
  return bf16 ? read_t<__nv_bfloat16>(c, bt, k, v, d, block, status, st)
              : read_t<float>(c, bt, k, v, d, block, status, st);
}

}  // namespace kv4
}  // namespace fvattn
