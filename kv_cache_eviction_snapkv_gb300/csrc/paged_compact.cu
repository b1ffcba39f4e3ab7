// Cut of a paged cache to its kept rows, in place.
//
// Per (layer, sequence, head) with n kept rows: the kept rows j < n stay where they are; the
// slots < n that no kept row holds (holes, ascending) take the kept rows j >= n (movers, in
// the list's order). As many holes as movers, and a mover's row lies at or behind n while a
// hole lies before it: no row that is read is written, so the moves need no order at all.
// That is the least traffic an in-place cut can have: each moved row read once and written
// once, the others not touched.
#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Exclusive prefix of `v` over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_prefix(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();                       // the sums of the call before have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return before + x - v;
}

// One block per (layer, sequence, head). Shared: the bitmap of kept rows < n, the movers'
// list entries and the holes' slots (16 bits each: max_keep <= 32768).
__global__ void __launch_bounds__(kThreads) paged_compact_kernel(const __grid_constant__ PagedCompactArgs a) {
  extern __shared__ uint32_t smem[];
  __shared__ int warp_sums[kWarps];
  __shared__ int bad;
  const int tid = threadIdx.x;
  const int64_t inst = blockIdx.x;
  const int h = (int)(inst % a.pv.Hkv);
  const int b = (int)(inst / a.pv.Hkv % a.S), layer = (int)(inst / a.pv.Hkv / a.S);
  const int max_rows = a.table_width << a.pv.page_shift;
  const int o0 = a.keep_offsets[b], o1 = a.keep_offsets[b + 1];
  const int len = a.lens[b], n = o1 - o0;
  if (o0 < 0 || o1 < o0 || o1 > a.keep_rows || n > a.max_keep || len < 0 || len > max_rows ||
      n > len) {
    if (tid == 0) record_status(a.status, KVSEL_ERR_BAD_INDEX);
    return;
  }
  const int words = (n + 31) >> 5;
  uint32_t* kept = smem;
  uint16_t* mover = reinterpret_cast<uint16_t*>(smem + ((a.max_keep + 31) >> 5));
  uint16_t* hole = mover + ((a.max_keep + 1) & ~1);
  const int32_t* trow = a.table + (int64_t)b * a.table_width;
  for (int w = tid; w < words; w += kThreads) kept[w] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  if (n < len) {
    for (int col = tid; col < (n + a.pv.page_size - 1) >> a.pv.page_shift; col += kThreads) {
      const int page = checked_page(a.pv, trow, col, a.status);
      if (page < 0) bad = 1;
      else if (a.ref && a.ref[page] > 1) {
        record_status(a.status, KVSEL_ERR_SHARED_PAGE);
        bad = 1;
      }
    }
  }
  const int32_t* list = a.keep_idx + ((int64_t)layer * a.keep_rows + o0) * a.pv.Hkv + h;
  int movers = 0;
  for (int s0 = 0; s0 < n; s0 += kThreads) {
    const int s = s0 + tid;
    int idx = 0;
    bool late = false;
    if (s < n) {
      idx = list[(int64_t)s * a.pv.Hkv];
      late = idx >= n;
      if (idx < 0 || idx >= len) {
        bad = 1;
        record_status(a.status, KVSEL_ERR_BAD_INDEX);
      } else if (late) {
        if (checked_page(a.pv, trow, idx >> a.pv.page_shift, a.status) < 0) bad = 1;
      } else if (atomicOr(&kept[idx >> 5], 1u << (idx & 31)) >> (idx & 31) & 1u) {
        bad = 1;                         // named twice
        record_status(a.status, KVSEL_ERR_BAD_INDEX);
      }
    }
    int total;
    const int at = movers + block_prefix(late, warp_sums, &total);
    if (late) mover[at] = (uint16_t)s;
    movers += total;
  }
  int holes = 0;
  for (int w0 = 0; w0 < words; w0 += kThreads) {
    const int w = w0 + tid;
    uint32_t free = 0;
    if (w < words) {
      free = ~kept[w];
      if (w == words - 1 && (n & 31)) free &= (1u << (n & 31)) - 1;
    }
    int total;
    int at = holes + block_prefix(__popc(free), warp_sums, &total);
    while (free) {
      hole[at++] = (uint16_t)(w * 32 + __ffs(free) - 1);
      free &= free - 1;
    }
    holes += total;
  }
  __syncthreads();
  if (bad) return;                       // uniform: set before the barriers above
  int32_t* pos = a.slot_pos ? a.slot_pos + ((int64_t)layer * a.keep_rows + o0) * a.pv.Hkv + h : nullptr;
  if (pos)
    for (int s = tid; s < n; s += kThreads)
      if (kept[s >> 5] >> (s & 31) & 1u) pos[(int64_t)s * a.pv.Hkv] = s;
  const int vecs = a.pv.head_units * 2;  // 16-byte vectors of a head's row
  const int64_t base = layer * a.pv.layer_bytes + (int64_t)h * a.pv.head_units * kRowUnit;
  for (int e = tid; e < holes * vecs; e += kThreads) {
    const int i = e / vecs, v = e - i * vecs;
    const int slot = hole[i], row = list[(int64_t)mover[i] * a.pv.Hkv];
    const int sp = trow[row >> a.pv.page_shift], dp = trow[slot >> a.pv.page_shift];
    const int64_t so = base + (int64_t)row_units(a.pv, sp, row & (a.pv.page_size - 1)) * kRowUnit + v * 16;
    const int64_t d0 = base + (int64_t)row_units(a.pv, dp, slot & (a.pv.page_size - 1)) * kRowUnit + v * 16;
    *reinterpret_cast<uint4*>(a.pv.k + d0) = *reinterpret_cast<const uint4*>(a.pv.k + so);
    *reinterpret_cast<uint4*>(a.pv.v + d0) = *reinterpret_cast<const uint4*>(a.pv.v + so);
    if (pos && v == 0) pos[(int64_t)slot * a.pv.Hkv] = row;
  }
}

}  // namespace

cudaError_t launch_paged_compact(const PagedCompactArgs& a) {
  auto lists = [](int n) { return ((n + 31) >> 5) * 4 + 2 * ((n + 1) & ~1) * 2; };
  const int smem = lists(a.max_keep);
  if (smem > 48 * 1024) {
    // always the same value: another thread's call may come between
    const cudaError_t e = cudaFuncSetAttribute(
        paged_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, lists(kMaxKeep));
    if (e) return e;
  }
  const int64_t insts = (int64_t)a.pv.layers * a.S * a.pv.Hkv;
  paged_compact_kernel<<<(unsigned)insts, kThreads, smem, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvsel
