// kv4_attn.cu -- attention over the 4-bit cache: one warp per (row, query head), one
// pass over the visible keys with the running maximum and sum of the softmax, fp32.
#include "kv4.cuh"

namespace fvattn {
namespace kv4 {

template <typename T, int HD>
__global__ void __launch_bounds__(128)
    attn_kernel(const Cache c, const Batch bt, const T* __restrict__ q, long long q_stride, int Hq,
                T* __restrict__ out, float* __restrict__ lse, float scale, int causal, int block,
                const int* __restrict__ kv_idx, const int* __restrict__ kv_cnt, int* status) {
  constexpr int C = HD / 32;   // channels per lane
  const long long unit = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit == 0 && lane == 0 && __ldg(bt.cu + bt.B) > bt.rows) record_status(status, FVATTN_ERR_INVALID_ARG);
  const int r = static_cast<int>(unit / Hq);
  const int hq = static_cast<int>(unit - static_cast<long long>(r) * Hq);
  if (r >= bt.rows) return;
  int b;
  if (!sequence_of(bt, r, b)) return;
  const int h = hq / (Hq / c.H);
  const int n = held(bt, b, block, status);
  const int pos = n - (__ldg(bt.cu + b + 1) - r);
  const int seen = causal ? min(max(pos + 1, 0), n) : n;
  const Layout L(HD, block);
  const float ks = scale * (c.k_scale ? __ldg(c.k_scale + h) : 1.f);
  float qv[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    qv[i] = static_cast<float>(q[static_cast<long long>(r) * q_stride + hq * HD + lane * C + i]) * ks;
    o[i] = 0.f;
  }
  const int pages = (seen + block - 1) / block;
  const int* list = kv_idx ? kv_idx + (static_cast<size_t>(r) * c.H + h) * bt.max_pages : nullptr;
  int cnt = pages, held_pages = (n + block - 1) / block, before = -1;
  if (list) {
    cnt = __ldg(kv_cnt + static_cast<size_t>(r) * c.H + h);
    if (cnt < 0 || cnt > bt.max_pages) {
      if (lane == 0) record_status(status, FVATTN_ERR_INVALID_ARG);
      cnt = min(max(cnt, 0), bt.max_pages);
    }
  }
  for (int e = 0; e < cnt; ++e) {
    int pg = e;
    if (list) {
      pg = __ldg(list + e);
      const bool good = pg > before && pg >= 0 && pg < held_pages;
      before = pg;
      if (!good) {
        if (lane == 0) record_status(status, FVATTN_ERR_INVALID_ARG);
        continue;
      }
    }
    if (pg >= pages) continue;
    const int slot = pool_slot(bt, c.num_pages, b, pg, status);
    if (slot < 0) continue;
    const uint8_t* rec = c.pages + (static_cast<size_t>(slot) * c.H + h) * L.rec;
    const int keys = min(block, seen - pg * block);
    for (int t = 0; t < keys; ++t) {
      const int ch = lane * C;
      auto value = [&](int codes, int scales, int i) {
        const uint8_t byte = rec[codes + t * (HD / 2) + ((ch + i) >> 1)];
        const uint32_t w = ((ch + i) & 1) ? byte >> 4 : byte & 15;
        uint32_t p[4];
        e2m1x8_to_half2(w, p);
        return __low2float(*reinterpret_cast<__half2*>(&p[0])) *
               e4m3_to_float(rec[scales + t * (HD / kGroup) + (ch + i) / kGroup]);
      };
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) s = fmaf(qv[i], value(0, L.kscale(), i), s);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      const float mn = fmaxf(m, s);
      const float f = __expf(m - mn), pr = __expf(s - mn);
      m = mn;
      l = l * f + pr;
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] = fmaf(pr, value(L.vcodes(), L.vscale(), i), o[i] * f);
    }
  }
  const float inv = l > 0.f ? (c.v_scale ? __ldg(c.v_scale + h) : 1.f) / l : 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) out[static_cast<size_t>(unit) * HD + lane * C + i] = static_cast<T>(o[i] * inv);
  if (lse && lane == 0) lse[unit] = l > 0.f ? m + logf(l) : -INFINITY;
}

cudaError_t launch_attn(const Cache& c, const Batch& bt, const void* q, long long q_stride, int Hq, void* out,
                        float* lse, bool bf16, float scale, int causal, int d, int block, const int* kv_idx,
                        const int* kv_cnt, int* status, cudaStream_t st) {
  const long long grid = (static_cast<long long>(bt.rows) * Hq + 3) / 4;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
#define FVATTN_KV4_ATTN(T, HD)                                                                                  \
  attn_kernel<T, HD><<<static_cast<unsigned>(grid), 128, 0, st>>>(c, bt, static_cast<const T*>(q), q_stride, Hq, \
                                                                  static_cast<T*>(out), lse, scale, causal,      \
                                                                  block, kv_idx, kv_cnt, status)
  if (bf16) {
    if (d == 128) FVATTN_KV4_ATTN(__nv_bfloat16, 128); else FVATTN_KV4_ATTN(__nv_bfloat16, 64);
  } else {
    if (d == 128) FVATTN_KV4_ATTN(float, 128); else FVATTN_KV4_ATTN(float, 64);
  }
#undef FVATTN_KV4_ATTN
  return cudaGetLastError();
}

}  // namespace kv4
}  // namespace fvattn
