// Descriptors and device helpers shared by the paged-cache kernels.
#pragma once

#include "kvsel_device.cuh"

namespace kvsel {

// Offset of row r of a page within its layer, in units of 32 bytes: they fit 32
// bits for pools of up to 128 GiB a layer (the host checks that).
__device__ __forceinline__ uint32_t row_units(const PagedView& pv, int page, int r) {
  return (uint32_t)page * pv.page_units + (uint32_t)r * pv.row_units;
}

// Page of column `col` of a sequence, or -1 (and BAD_INDEX) if it is not one
// of the pool's.
__device__ __forceinline__ int checked_page(const PagedView& pv, const int32_t* table_row, int col,
                                            int* status) {
  const int page = __ldg(table_row + col);
  if (page >= 0 && page < pv.num_pages) return page;
  record_status(status, KVSEL_ERR_BAD_INDEX);
  return -1;
}

// Length of a sequence, held to [0, max_rows].
__device__ __forceinline__ int checked_len(int len, int max_rows, int* status) {
  if (len >= 0 && len <= max_rows) return len;
  record_status(status, KVSEL_ERR_BAD_INDEX);
  return len < 0 ? 0 : max_rows;
}

// x / y, x >= 0, y > 0: mostly small, and a division of 32 bits is several times cheaper.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return (x | y) >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}

// Two fp32 values and the instructions on them.
struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(Two x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

}  // namespace kvsel
