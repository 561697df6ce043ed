// kv4_api.cu -- the extern "C" entry points of the paged 4-bit key/value cache
// (declared in include/fvattn.h): host-side validation, workspace layout, dispatch.
// No entry point allocates device memory or synchronizes the host.
#include <atomic>
#include <chrono>
#include <cmath>

#include "kv4.cuh"

namespace fvattn {
namespace kv4 {
cudaError_t launch_append(const Cache& c, const Batch& bt, const void* k, const void* v, long long ks,
                          long long vs, bool bf16, int d, int block, const Status& status, cudaStream_t st);
cudaError_t launch_read(const Cache& c, const Batch& bt, void* k, void* v, bool bf16, int d, int block,
                        const Status& status, cudaStream_t st);
cudaError_t launch_select(const Cache& c, const Batch& bt, const void* q, long long q_stride, int Hq, bool bf16,
                          float scale, float p, int k_min, int d, int block, int* kv_idx, int* kv_cnt,
                          const Status& status, cudaStream_t st);
cudaError_t launch_attn(const Cache& c, const Batch& bt, const void* q, long long q_stride, int Hq, void* out,
                        float* lse, bool bf16, float scale, int causal, int d, int block, int max_q, const int* kv_idx,
                        const int* kv_cnt, const Status& status, uint8_t* ws, int num_sms, cudaStream_t st);
size_t attn_ws_bytes(int d, int max_q, int G);
size_t attn_ws_clear();
}  // namespace kv4
}  // namespace fvattn

namespace {

using fvattn::kWsHeaderBytes;

constexpr int kMaxHeads = 4096;
constexpr int kMaxGroup = 64;          // query heads per KV head
constexpr int kMaxSelectPages = 8192;  // a row's masses live in shared memory
constexpr long long kMaxTokens = 1ll << 30;
constexpr int kMaxRows = 1 << 24;
constexpr int kMaxBatch = 1 << 20;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

bool valid_sizes(const fvattn_kv4_cache* c, const fvattn_kv4_batch* b) {
  if (!c || !b) return false;
  if (c->num_pages < 1 || c->H < 1 || c->H > kMaxHeads) return false;
  if ((c->d != 64 && c->d != 128) || (c->block != 64 && c->block != 128)) return false;
  if (b->B < 1 || b->B > kMaxBatch || b->max_pages < 1 || b->rows < 0 || b->rows > kMaxRows || b->max_q < 1)
    return false;
  if (static_cast<long long>(b->rows) * c->H > 0x3FFFFFFFll) return false;   // (row, KV head) pairs are ints
  return static_cast<long long>(b->max_pages) * c->block <= kMaxTokens;
}

bool valid_heads(const fvattn_kv4_cache* c, int Hq) {
  return Hq >= c->H && Hq <= kMaxHeads && Hq % c->H == 0 && Hq / c->H <= kMaxGroup;
}

bool valid_pointers(const fvattn_kv4_cache* c, const fvattn_kv4_batch* b) {
  if (!c->pages || !aligned(c->pages, 16) || !aligned(c->ksum, 16)) return false;
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return false;
  if (!b->table || !b->kv_len || !b->cu) return false;
  return aligned(b->table, 4) && aligned(b->kv_len, 4) && aligned(b->cu, 4);
}

// Bytes of a [rows, H, d] tensor with the given row stride; 0 if the stride is invalid.
size_t strided_bytes(long long rows, int heads, int d, int64_t stride, int es, bool* ok) {
  const int64_t row = static_cast<int64_t>(heads) * d;
  *ok = stride >= row && stride <= (1ll << 31) && (stride * es) % 16 == 0;
  if (!*ok || rows == 0) return 0;
  return (static_cast<size_t>(rows - 1) * stride + row) * es;
}

bool valid_dtype(fvattn_dtype dt) { return dt == FVATTN_BF16 || dt == FVATTN_FP32; }

fvattn::kv4::Cache cache_of(const fvattn_kv4_cache* c) {
  return fvattn::kv4::Cache{static_cast<uint8_t*>(c->pages), c->ksum, c->k_scale, c->v_scale, c->num_pages, c->H};
}
fvattn::kv4::Batch batch_of(const fvattn_kv4_batch* b) {
  return fvattn::kv4::Batch{b->table, b->kv_len, b->cu, b->B, b->max_pages, b->rows};
}
size_t pool_bytes(const fvattn_kv4_cache* c) {
  return static_cast<size_t>(c->num_pages) * c->H * c->block * (c->d + c->d / 8);
}

__global__ void clear_kernel(uint4* p, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// Where the calls' numbers start: somewhere else in every process and every copy of the library, so
// that memory which another one's calls have left flags in does not carry the numbers of this one's.
unsigned long long first_number() {
  unsigned long long x = static_cast<unsigned long long>(std::chrono::system_clock::now().time_since_epoch().count());
  x ^= static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(&first_number)) << 20;
  x *= 0x9E3779B97F4A7C15ull;                 // 2^64 / golden ratio: all bits reach the upper ones
  return 1ull + (x >> 17);                    // 1 .. 2^47
}

// Workspace check, and the call's number (kv4.cuh). The header and `clear` bytes of counters behind
// it are cleared only where that does not do: in a captured call, whose replays share the number,
// and in a call without rows, which runs no other kernel. A clearing launch costs 2 us of host time
// and 1 us of the stream; it is a kernel because a memset between two kernels costs 3 us.
fvattn_status begin(void* ws, size_t have, size_t need, cudaStream_t st, int rows, fvattn::kv4::Status* status,
                    size_t clear = 0) {
  if (!ws || !aligned(ws, 256) || have < need) return FVATTN_ERR_WORKSPACE;
  static std::atomic<unsigned long long> calls{first_number()};
  status->h = static_cast<fvattn::WsHeader*>(ws);
  status->call = calls.fetch_add(1, std::memory_order_relaxed) & 0xFFFFFFFFFFFFull;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  const bool known = cudaStreamIsCapturing(st, &cap) == cudaSuccess;
  if (!known) cudaGetLastError();
  if (known && cap == cudaStreamCaptureStatusNone && rows > 0) return FVATTN_OK;
  clear_kernel<<<1, 512, 0, st>>>(static_cast<uint4*>(ws), static_cast<int>((kWsHeaderBytes + clear) / 16));
  return cudaGetLastError() == cudaSuccess ? FVATTN_OK : FVATTN_ERR_CUDA;
}

// SM count of the current device, kept after the first look-up (every writer of an entry stores
// the same value, so calls from several host threads may race to fill it).
int device_sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) {
    const int n = cache[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

fvattn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FVATTN_OK : FVATTN_ERR_CUDA; }

}  // namespace

extern "C" {

size_t fvattn_kv4_workspace_bytes(fvattn_op op, const fvattn_kv4_cache* cache, const fvattn_kv4_batch* batch,
                                  int Hq) {
  if (!valid_sizes(cache, batch)) return 0;
  switch (op) {
    case FVATTN_OP_KV4_APPEND:
    case FVATTN_OP_KV4_READ: return kWsHeaderBytes;
    case FVATTN_OP_KV4_SELECT:
      return valid_heads(cache, Hq) && batch->max_pages <= kMaxSelectPages ? kWsHeaderBytes : 0;
    case FVATTN_OP_KV4_ATTN:
      if (!valid_heads(cache, Hq)) return 0;
      return kWsHeaderBytes + fvattn::align_up(fvattn::kv4::attn_ws_bytes(cache->d, batch->max_q, Hq / cache->H), 256);
    default: return 0;
  }
}

fvattn_status fvattn_kv4_append(const fvattn_kv4_cache* cache, const fvattn_kv4_batch* batch, const void* k,
                                const void* v, int64_t k_stride, int64_t v_stride, fvattn_dtype dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_sizes(cache, batch) || !valid_pointers(cache, batch) || !valid_dtype(dtype))
    return FVATTN_ERR_INVALID_ARG;
  const bool any = batch->rows > 0;   // tensors without rows may be null
  if ((any && (!k || !v)) || !aligned(k, 16) || !aligned(v, 16)) return FVATTN_ERR_INVALID_ARG;
  const int es = dtype == FVATTN_BF16 ? 2 : 4;
  bool okk, okv;
  const size_t nk = strided_bytes(batch->rows, cache->H, cache->d, k_stride, es, &okk);
  const size_t nv = strided_bytes(batch->rows, cache->H, cache->d, v_stride, es, &okv);
  if (!okk || !okv) return FVATTN_ERR_INVALID_ARG;
  const size_t np = pool_bytes(cache);
  if (overlap(k, nk, cache->pages, np) || overlap(v, nv, cache->pages, np)) return FVATTN_ERR_INVALID_ARG;
  auto st = static_cast<cudaStream_t>(stream);
  fvattn::kv4::Status status;
  const fvattn_status s = begin(workspace, workspace_bytes, kWsHeaderBytes, st, batch->rows, &status);
  if (s != FVATTN_OK || batch->rows == 0) return s;
  return from_cuda(fvattn::kv4::launch_append(cache_of(cache), batch_of(batch), k, v, k_stride, v_stride,
                                              dtype == FVATTN_BF16, cache->d, cache->block, status, st));
}

fvattn_status fvattn_kv4_read(const fvattn_kv4_cache* cache, const fvattn_kv4_batch* batch, void* k_out,
                              void* v_out, fvattn_dtype dtype, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (!valid_sizes(cache, batch) || !valid_pointers(cache, batch) || !valid_dtype(dtype))
    return FVATTN_ERR_INVALID_ARG;
  const bool any = batch->rows > 0;
  if ((any && (!k_out || !v_out)) || !aligned(k_out, 16) || !aligned(v_out, 16)) return FVATTN_ERR_INVALID_ARG;
  const size_t no = static_cast<size_t>(batch->rows) * cache->H * cache->d * (dtype == FVATTN_BF16 ? 2 : 4);
  const size_t np = pool_bytes(cache);
  if (overlap(k_out, no, v_out, no) || overlap(k_out, no, cache->pages, np) || overlap(v_out, no, cache->pages, np))
    return FVATTN_ERR_INVALID_ARG;
  auto st = static_cast<cudaStream_t>(stream);
  fvattn::kv4::Status status;
  const fvattn_status s = begin(workspace, workspace_bytes, kWsHeaderBytes, st, batch->rows, &status);
  if (s != FVATTN_OK || batch->rows == 0) return s;
  return from_cuda(fvattn::kv4::launch_read(cache_of(cache), batch_of(batch), k_out, v_out, dtype == FVATTN_BF16,
                                            cache->d, cache->block, status, st));
}

fvattn_status fvattn_kv4_select(const fvattn_kv4_cache* cache, const fvattn_kv4_batch* batch, const void* q,
                                int64_t q_stride, int Hq, fvattn_dtype dtype, float scale, float p, int k_min,
                                int32_t* kv_idx, int32_t* kv_cnt, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!valid_sizes(cache, batch) || !valid_pointers(cache, batch) || !valid_dtype(dtype) || !cache->ksum)
    return FVATTN_ERR_INVALID_ARG;
  const bool any = batch->rows > 0;
  if ((any && (!q || !kv_idx || !kv_cnt)) || !aligned(q, 16) || !aligned(kv_idx, 4) || !aligned(kv_cnt, 4))
    return FVATTN_ERR_INVALID_ARG;
  if (!valid_heads(cache, Hq) || batch->max_pages > kMaxSelectPages) return FVATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale) || !(p > 0.f && p <= 1.f) || k_min < 1) return FVATTN_ERR_INVALID_ARG;
  bool ok;
  strided_bytes(batch->rows, Hq, cache->d, q_stride, dtype == FVATTN_BF16 ? 2 : 4, &ok);
  if (!ok) return FVATTN_ERR_INVALID_ARG;
  const size_t need = fvattn_kv4_workspace_bytes(FVATTN_OP_KV4_SELECT, cache, batch, Hq);
  auto st = static_cast<cudaStream_t>(stream);
  fvattn::kv4::Status status;
  const fvattn_status s = begin(workspace, workspace_bytes, need, st, batch->rows, &status);
  if (s != FVATTN_OK || batch->rows == 0) return s;
  return from_cuda(fvattn::kv4::launch_select(cache_of(cache), batch_of(batch), q, q_stride, Hq,
                                              dtype == FVATTN_BF16, scale, p, k_min, cache->d, cache->block, kv_idx, kv_cnt, status, st));
}

fvattn_status fvattn_kv4_attn(const fvattn_kv4_cache* cache, const fvattn_kv4_batch* batch, const void* q,
                              int64_t q_stride, int Hq, void* out, float* lse, fvattn_dtype dtype, float scale,
                              int causal, const int32_t* kv_idx, const int32_t* kv_cnt, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!valid_sizes(cache, batch) || !valid_pointers(cache, batch) || !valid_dtype(dtype))
    return FVATTN_ERR_INVALID_ARG;
  const bool any = batch->rows > 0;
  if ((any && (!q || !out)) || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return FVATTN_ERR_INVALID_ARG;
  if ((any && (kv_idx == nullptr) != (kv_cnt == nullptr)) || !aligned(kv_idx, 4) || !aligned(kv_cnt, 4))
    return FVATTN_ERR_INVALID_ARG;
  if (!valid_heads(cache, Hq) || !(scale > 0.f) || !std::isfinite(scale)) return FVATTN_ERR_INVALID_ARG;
  const int es = dtype == FVATTN_BF16 ? 2 : 4;
  bool ok;
  const size_t nq = strided_bytes(batch->rows, Hq, cache->d, q_stride, es, &ok);
  const size_t no = static_cast<size_t>(batch->rows) * Hq * cache->d * es;
  if (!ok || overlap(q, nq, out, no) || overlap(out, no, cache->pages, pool_bytes(cache))) return FVATTN_ERR_INVALID_ARG;
  const size_t need = fvattn_kv4_workspace_bytes(FVATTN_OP_KV4_ATTN, cache, batch, Hq);
  auto st = static_cast<cudaStream_t>(stream);
  fvattn::kv4::Status status;
  const fvattn_status s = begin(workspace, workspace_bytes, need, st, batch->rows, &status,
                                fvattn::kv4::attn_ws_clear());
  if (s != FVATTN_OK || batch->rows == 0) return s;
  const int sms = device_sm_count();
  if (sms <= 0) return FVATTN_ERR_CUDA;
  return from_cuda(fvattn::kv4::launch_attn(cache_of(cache), batch_of(batch), q, q_stride, Hq, out, lse,
                                            dtype == FVATTN_BF16, scale, causal != 0, cache->d, cache->block,
                                            batch->max_q, kv_idx, kv_cnt, status,
                                            static_cast<uint8_t*>(workspace) + kWsHeaderBytes, sms, st));
}

}  // extern "C"
