// kv4_select.cu -- the pages a row attends: softmax over the mean keys of the full
// pages before the row's own, averaged over the query heads of a KV head, then Top-p
// with a Top-k floor.
//
// All arithmetic is fp64: the page sums are exact integers, so a score differs from
// its definition by a few 2^-53 and only true ties are decided by rounding.
#include "kv4.cuh"

namespace fvattn {
namespace kv4 {

constexpr int kSelThreads = 256;

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

__device__ __forceinline__ double block_reduce(double v, bool max, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double u = __shfl_xor_sync(0xffffffffu, v, o);
    v = max ? fmax(v, u) : v + u;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < kSelThreads / 32; ++i) v = max ? fmax(v, red[i]) : v + red[i];
  return v;
}

// One block per (row, KV head). Shared memory: scores and masses [n2] fp64, order [n2].
template <typename T, int HD>
__global__ void __launch_bounds__(kSelThreads)
    select_kernel(const Cache c, const Batch bt, const T* __restrict__ q, long long q_stride, int G, double w,
                  float p, int k_min, int block, int n2, int* __restrict__ kv_idx, int* __restrict__ kv_cnt,
                  int* status) {
  extern __shared__ double sh[];
  double* x = sh;                 // scores of one query head
  double* mass = sh + n2;
  int* order = reinterpret_cast<int*>(sh + 2 * n2);
  __shared__ double red[kSelThreads / 32];
  __shared__ int s_cnt;
  const int r = blockIdx.x / c.H, h = blockIdx.x % c.H;
  if (blockIdx.x == 0 && threadIdx.x == 0 && __ldg(bt.cu + bt.B) > bt.rows)
    record_status(status, FVATTN_ERR_INVALID_ARG);
  int b;
  if (!sequence_of(bt, r, b)) return;
  const int n = held(bt, b, block, status);
  const int pos = n - (__ldg(bt.cu + b + 1) - r);
  const size_t unit = static_cast<size_t>(r) * c.H + h;
  int* out = kv_idx + unit * bt.max_pages;
  if (pos < 0 || pos >= n) {
    if (threadIdx.x == 0) {
      record_status(status, FVATTN_ERR_INVALID_ARG);
      kv_cnt[unit] = 0;
    }
    return;
  }
  const int o = pos / block;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (c.k_scale) w *= static_cast<double>(__ldg(c.k_scale + h));
  for (int j = threadIdx.x; j < n2; j += kSelThreads) mass[j] = j < o ? 0.0 : -1.0;
  for (int g = 0; g < G; ++g) {
    const T* qr = q + static_cast<long long>(r) * q_stride + (static_cast<long long>(h) * G + g) * HD;
    double qv[HD / 32];
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) qv[i] = static_cast<double>(to_float(qr[i * 32 + lane]));
    double mx = -INFINITY;
    for (int j = warp; j < o; j += kSelThreads / 32) {
      const int slot = pool_slot(bt, c.num_pages, b, j, status);
      double s = 0.0;
      if (slot >= 0) {
        const int* ks = c.ksum + (static_cast<size_t>(slot) * c.H + h) * HD;
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) s += qv[i] * static_cast<double>(__ldg(ks + i * 32 + lane));
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= w;
      if (lane == 0) x[j] = s;
      mx = fmax(mx, s);
    }
    mx = block_reduce(mx, true, red);
    double z = 0.0;
    for (int j = threadIdx.x; j < o; j += kSelThreads) {
      x[j] = exp(x[j] - mx);
      z += x[j];
    }
    z = block_reduce(z, false, red);
    for (int j = threadIdx.x; j < o; j += kSelThreads) mass[j] += x[j] / z;
    __syncthreads();
  }
  for (int j = threadIdx.x; j < n2; j += kSelThreads) {
    if (j < o) mass[j] /= G;
    order[j] = j;
  }
  // descending mass, ties by the lower page
  for (int size = 2; size <= n2; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      __syncthreads();
      for (int t = threadIdx.x; t < n2 / 2; t += kSelThreads) {
        const int lo = 2 * t - (t & (stride - 1)), hi = lo + stride;
        const bool desc = (lo & size) == 0;
        const double a = mass[lo], e = mass[hi];
        const bool less = a < e || (a == e && order[lo] > order[hi]);
        if (less == desc) {
          mass[lo] = e; mass[hi] = a;
          const int i = order[lo]; order[lo] = order[hi]; order[hi] = i;
        }
      }
    }
  __syncthreads();
  if (threadIdx.x == 0) {
    int np = o;
    if (p < 1.f) {
      double acc = 0.0;
      for (int j = 0; j < o; ++j) {
        acc += mass[j];
        if (acc >= static_cast<double>(p)) { np = j + 1; break; }
      }
    }
    s_cnt = min(o, max(np, k_min));
  }
  __syncthreads();
  const int cnt = s_cnt;
  for (int j = threadIdx.x; j < n2; j += kSelThreads) x[j] = 0.0;
  __syncthreads();
  for (int j = threadIdx.x; j < cnt; j += kSelThreads) x[order[j]] = 1.0;
  __syncthreads();
  if (threadIdx.x == 0) {
    int m = 0;
    for (int j = 0; j < o; ++j)
      if (x[j] != 0.0) out[m++] = j;
    out[m++] = o;
    kv_cnt[unit] = m;
  }
}

template <typename T, int HD>
static cudaError_t select_t(const Cache& c, const Batch& bt, const void* q, long long q_stride, int G, double w,
                            float p, int k_min, int block, int* kv_idx, int* kv_cnt, int* status,
                            cudaStream_t st) {
  int n2 = 2;
  while (n2 < bt.max_pages) n2 <<= 1;
  const int smem = n2 * 20;
  const long long grid = static_cast<long long>(bt.rows) * c.H;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(select_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  select_kernel<T, HD><<<static_cast<unsigned>(grid), kSelThreads, smem, st>>>(
      c, bt, static_cast<const T*>(q), q_stride, G, w, p, k_min, block, n2, kv_idx, kv_cnt, status);
  return cudaGetLastError();
}

cudaError_t launch_select(const Cache& c, const Batch& bt, const void* q, long long q_stride, int Hq, bool bf16,
                          float scale, float p, int k_min, int d, int block, int* kv_idx, int* kv_cnt,
                          int* status, cudaStream_t st) {
  const int G = Hq / c.H;
  const double w = static_cast<double>(scale) / (1024.0 * block);
  if (d == 128)
    return bf16 ? select_t<__nv_bfloat16, 128>(c, bt, q, q_stride, G, w, p, k_min, block, kv_idx, kv_cnt, status, st)
                : select_t<float, 128>(c, bt, q, q_stride, G, w, p, k_min, block, kv_idx, kv_cnt, status, st);
  return bf16 ? select_t<__nv_bfloat16, 64>(c, bt, q, q_stride, G, w, p, k_min, block, kv_idx, kv_cnt, status, st)
              : select_t<float, 64>(c, bt, q, q_stride, G, w, p, k_min, block, kv_idx, kv_cnt, status, st);
}

}  // namespace kv4
}  // namespace fvattn
