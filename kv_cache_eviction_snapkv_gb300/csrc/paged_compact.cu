// Cut of a paged cache to its kept rows, in place.
//
// Per (layer, sequence, head) with n kept rows: the kept rows j < n stay where they are; the
// slots < n that no kept row holds (holes, ascending) take the kept rows j >= n (movers, in
// the list's order). As many holes as movers, and a mover's row lies at or behind n while a
// hole lies before it: no row that is read is written, so the moves need no order at all.
// That is the least traffic an in-place cut can have: each moved row read once and written
// once, the others not touched.
//
// Bound by memory for a long list, by the plan's chain of loads and barriers for a short one.
// The plan (who moves where) needs the instance's whole list, so it is made by the block that
// uses it, in shared memory: a bitmap of the kept rows < n, the movers by a prefix count over
// the list, the holes by one over the bitmap. Where instances are few, several blocks make the
// same plan and share out the moves; that costs less than a plan kept in memory and a second
// launch.
//
// Measured: 32 layers x 8 heads cut from 16384 rows to 2048, 474 MB: 85 us, 5.6 TB/s, 82% of the
// copy bandwidth; 126 short instances: 10 us.
#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 8;            // list entries a thread has in flight
constexpr int kChunk = 1024;         // moves whose row offsets are in shared memory at a time
constexpr int kAhead = 4;            // 16-byte vectors a thread moves at a time, of K and of V

// Prefix count of flags over kBatch rounds of the block's threads, round-major (thread t of round
// i comes before thread 0 of round i + 1): before[i] gets the flags before this thread's, the
// return value is their number.
__device__ __forceinline__ int batch_prefix(const bool (&flag)[kBatch], int (&before)[kBatch],
                                            int (*counts)[kWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  static_assert(kBatch * kWarps == 64, "two counts a lane");
  uint32_t mask[kBatch];
  __syncthreads();                   // the counts of the call before have been read
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    mask[i] = __ballot_sync(0xffffffffu, flag[i]);
    if (lane == 0) counts[i][warp] = __popc(mask[i]);
  }
  __syncthreads();
  const int2 c = reinterpret_cast<const int2*>(&counts[0][0])[lane];
  int x = c.x + c.y;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int at = i * kWarps + warp;                          // this warp's count, among the 64
    const int upto = __shfl_sync(0xffffffffu, x, at >> 1);     // inclusive of the pair
    const int pair_y = __shfl_sync(0xffffffffu, c.y, at >> 1);
    const int own = __popc(mask[i]);
    before[i] = upto - (at & 1 ? own : own + pair_y) + __popc(mask[i] & ((1u << lane) - 1));
  }
  return __shfl_sync(0xffffffffu, x, 31);
}

// Blocks (layer, sequence, head) x parts. Shared: the movers' rows, the bitmap of kept rows < n
// and the holes' slots (16 bits: max_keep <= 32768).
__global__ void __launch_bounds__(kThreads, 4) paged_compact_kernel(const __grid_constant__ PagedCompactArgs a,
                                                                    int parts) {
  extern __shared__ uint32_t smem[];
  __shared__ __align__(8) int counts[kBatch][kWarps];
  __shared__ uint32_t from[kChunk], to[kChunk];
  __shared__ int bad;
  const int tid = threadIdx.x;
  const int64_t inst = blockIdx.x / parts;
  const int part = (int)(blockIdx.x - inst * parts);
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
  int* mover = reinterpret_cast<int*>(smem);
  uint32_t* kept = smem + a.max_keep;
  uint16_t* hole = reinterpret_cast<uint16_t*>(kept + ((a.max_keep + 31) >> 5));
  const int32_t* trow = a.table + (int64_t)b * a.table_width;
  for (int w = tid; w < words; w += kThreads) kept[w] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  const int32_t* list = a.keep_idx + ((int64_t)layer * a.keep_rows + o0) * a.pv.Hkv + h;
  int movers = 0;
  for (int s0 = 0; s0 < n; s0 += kThreads * kBatch) {
    int idx[kBatch], page[kBatch], at[kBatch];
    bool late[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + i * kThreads + tid;
      idx[i] = s < n ? list[(int64_t)s * a.pv.Hkv] : 0;
    }
    if (s0 == 0 && n < len) {            // while the list arrives: the pages that may be written
      for (int col = tid; col < (n + a.pv.page_size - 1) >> a.pv.page_shift; col += kThreads) {
        const int p = checked_page(a.pv, trow, col, a.status);
        if (p < 0) {
          bad = 1;
        } else if (a.ref && a.ref[p] > 1) {
          record_status(a.status, KVSEL_ERR_SHARED_PAGE);
          bad = 1;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      late[i] = s0 + i * kThreads + tid < n && idx[i] >= n;
      page[i] = late[i] && idx[i] < len ? __ldg(trow + (idx[i] >> a.pv.page_shift)) : 0;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s0 + i * kThreads + tid >= n) continue;
      // out of range, on a page out of range, or named twice
      if (idx[i] < 0 || idx[i] >= len || (late[i] && (page[i] < 0 || page[i] >= a.pv.num_pages)) ||
          (!late[i] && (atomicOr(&kept[idx[i] >> 5], 1u << (idx[i] & 31)) >> (idx[i] & 31) & 1u))) {
        bad = 1;
        record_status(a.status, KVSEL_ERR_BAD_INDEX);
      }
    }
    const int total = batch_prefix(late, at, counts);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (late[i]) mover[movers + at[i]] = idx[i];
    movers += total;
  }
  __syncthreads();                       // the bitmap is whole
  int holes = 0;
  for (int s0 = 0; s0 < n; s0 += kThreads * kBatch) {
    int at[kBatch];
    bool gap[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + i * kThreads + tid;
      gap[i] = s < n && !(kept[s >> 5] >> (s & 31) & 1u);
    }
    const int total = batch_prefix(gap, at, counts);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (gap[i]) hole[holes + at[i]] = (uint16_t)(s0 + i * kThreads + tid);
    holes += total;
  }
  __syncthreads();
  if (bad) return;                       // uniform; holes == movers from here on
  int32_t* pos = a.slot_pos ? a.slot_pos + ((int64_t)layer * a.keep_rows + o0) * a.pv.Hkv + h : nullptr;
  if (pos)
    for (int s = part * kThreads + tid; s < n; s += parts * kThreads)
      if (kept[s >> 5] >> (s & 31) & 1u) pos[(int64_t)s * a.pv.Hkv] = s;

  const int vec_shift = a.pv.head_units == 16 ? 5 : a.pv.head_units == 8 ? 4 : 3;  // vectors of a head
  const int64_t base = layer * a.pv.layer_bytes + (int64_t)h * a.pv.head_units * kRowUnit;
  char* kb = a.pv.k + base;
  char* vb = a.pv.v + base;
  const int m0 = (int)((int64_t)holes * part / parts), m1 = (int)((int64_t)holes * (part + 1) / parts);
  for (int c0 = m0; c0 < m1; c0 += kChunk) {
    const int c = min(kChunk, m1 - c0);
    for (int i = tid; i < c; i += kThreads) {
      const int slot = hole[c0 + i], row = mover[c0 + i];
      from[i] = row_units(a.pv, trow[row >> a.pv.page_shift], row & (a.pv.page_size - 1));
      to[i] = row_units(a.pv, trow[slot >> a.pv.page_shift], slot & (a.pv.page_size - 1));
      if (pos) pos[(int64_t)slot * a.pv.Hkv] = row;
    }
    __syncthreads();
    const int vecs = c << vec_shift;
    for (int e0 = tid; e0 < vecs; e0 += kThreads * kAhead) {
      uint4 k[kAhead], v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int e = e0 + u * kThreads;
        if (e < vecs) {
          const int64_t off = (int64_t)from[e >> vec_shift] * kRowUnit + (e & ((1 << vec_shift) - 1)) * 16;
          k[u] = __ldcs(reinterpret_cast<const uint4*>(kb + off));
          v[u] = __ldcs(reinterpret_cast<const uint4*>(vb + off));
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int e = e0 + u * kThreads;
        if (e < vecs) {
          const int64_t off = (int64_t)to[e >> vec_shift] * kRowUnit + (e & ((1 << vec_shift) - 1)) * 16;
          *reinterpret_cast<uint4*>(kb + off) = k[u];
          *reinterpret_cast<uint4*>(vb + off) = v[u];
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_paged_compact(const PagedCompactArgs& a) {
  static_assert((kMaxKeep / 32) * 4 + 6 * kMaxKeep + 2 * kChunk * 4 + 1024 <= 227 * 1024,
                "lists and offsets fit shared memory");
  auto lists = [](int n) { return n * 4 + ((n + 31) >> 5) * 4 + ((n + 1) & ~1) * 2; };
  const int smem = lists(a.max_keep);
  if (smem > 32 * 1024) {
    // always the same value: another thread's call may come between
    const cudaError_t e = cudaFuncSetAttribute(
        paged_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, lists(kMaxKeep));
    if (e) return e;
  }
  // blocks an instance: twelve an SM in all (four at a time: the plans of later ones then run
  // beside the moves of earlier ones; 85 us for a whole prompt, 88 with four), with 256 kept rows
  // or more each
  const int64_t insts = (int64_t)a.pv.layers * a.S * a.pv.Hkv;
  int64_t parts = 12 * (int64_t)a.sm_count / insts;
  if (parts > (a.max_keep + 255) / 256) parts = (a.max_keep + 255) / 256;
  if (parts < 1) parts = 1;
  paged_compact_kernel<<<(unsigned)(insts * parts), kThreads, smem, a.stream>>>(a, (int)parts);
  return cudaGetLastError();
}

}  // namespace kvsel
