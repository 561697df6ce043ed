// kv4.cuh -- shared definitions of the paged 4-bit key/value cache: record layout,
// the rows of a call, code conversions.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace fvattn {
namespace kv4 {

constexpr int kGroup = 16;   // channels that share a scale

// Byte offsets inside the record of one (page, KV head).
struct Layout {
  int codes, scales, rec;    // bytes of K codes, of K scales, of the record
  __host__ __device__ constexpr Layout(int d, int block)
      : codes(block * d / 2), scales(block * d / kGroup), rec(block * (d + d / 8)) {}
  __host__ __device__ constexpr int kscale() const { return codes; }
  __host__ __device__ constexpr int vcodes() const { return codes + scales; }
  __host__ __device__ constexpr int vscale() const { return 2 * codes + scales; }
};

struct Cache {
  uint8_t* pages;
  int32_t* ksum;
  const float* k_scale;
  const float* v_scale;
  int num_pages, H;
};

struct Batch {
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  int B, max_pages, rows;
};

// Where a call's kernels record errors. Every call has a number of its own, so nothing has to be
// cleared before it: what other calls have left in the workspace does not carry its number.
// (Replays of a captured call share theirs; there a kernel clears the words first.)
struct Status {
  WsHeader* h;
  unsigned long long call;   // 1 .. 2^48 - 1
};

// Names the call in the workspace; by one thread of the grid.
__device__ __forceinline__ void open_call(const Status& s) {
  if (blockIdx.x == 0 && threadIdx.x == 0) s.h->call = s.call;
}

// The call's first error stays.
__device__ __forceinline__ void record_status(const Status& s, int code) {
  unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(&s.h->record);
  while ((old >> 8) != s.call) {
    const unsigned long long seen = atomicCAS(&s.h->record, old, s.call << 8 | static_cast<unsigned>(code));
    if (seen == old) return;
    old = seen;
  }
}

// A sequence's length n, clamped to what its table row can hold. Positions count from the length
// itself (start_of): a row behind the table's end is left out, the others stay where they are.
__device__ __forceinline__ int held(int n, const Batch& bt, int block, const Status& status) {
  const int most = bt.max_pages * block;
  if (n < 0 || n > most) {
    record_status(status, FVATTN_ERR_INVALID_ARG);
    return min(max(n, 0), most);
  }
  return n;
}

// Where the call's rows end: those behind belong to no sequence.
__device__ __forceinline__ int rows_end(const Batch& bt, const int* cu) { return min(cu[bt.B], bt.rows); }

// Records row starts that are negative or fall, and an end outside the tensors; by one block, all its
// threads. cu: bt.cu or a copy.
__device__ __forceinline__ void check_rows(const Batch& bt, const int* cu, const Status& status) {
  if (blockIdx.x != 0) return;
  bool bad = threadIdx.x == 0 && (cu[bt.B] < 0 || cu[bt.B] > bt.rows);
  for (int b = threadIdx.x; b < bt.B; b += blockDim.x) bad |= cu[b] < 0 || (b + 1 < bt.B && cu[b + 1] < cu[b]);
  if (bad) record_status(status, FVATTN_ERR_INVALID_ARG);
}

// Position of the first of a sequence's q >= 0 rows, of n tokens.
__device__ __forceinline__ int start_of(int n, int q) { return max(n, 0) - q; }

// Pool slot of page pg (in [0, max_pages)) of sequence b; -1 (recorded) if invalid.
__device__ __forceinline__ int pool_slot(const Batch& bt, int num_pages, int b, int pg, const Status& status) {
  const int s = __ldg(bt.table + static_cast<size_t>(b) * bt.max_pages + pg);
  if (s < 0 || s >= num_pages) {
    record_status(status, FVATTN_ERR_INVALID_ARG);
    return -1;
  }
  return s;
}

// Eight E2M1 codes (one 32-bit word, lowest channel in the low bits) to four f16 pairs.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Eight fp32 values to E2M1 codes, x[0] in the lowest bits (nearest even, saturating at 6).
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// One E4M3 code to fp32 (exact).
__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
  uint32_t r;
  const uint16_t h = static_cast<uint16_t>(code & 0xFFu);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(r & 0xFFFFu)));
}

// Nearest E4M3 code of a non-negative fp32 value (ties to even, saturating at 448).
__device__ __forceinline__ uint32_t float_to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}

}  // namespace kv4
}  // namespace fvattn
