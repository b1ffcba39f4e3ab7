// One step of a page pool's bookkeeping: fork, reorder, grow, cut and free sequences.
//
// New sequence b continues the first m = min(old length, new length) rows of its parent. Its
// columns are: whole pages (column < m / page_size, shared), one started page (m % page_size
// rows), fresh pages up to the new length. Counting the whole uses of every page first makes
// the rest independent of any order: a started page stays with its lowest user if its count
// is 0 and is copied for the others; the pages with count 0 after that are free and go out,
// lowest first, in the order of (sequence, column). A page that is copied from always keeps
// a holder, so it is never handed out in the same step.
#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Workspace: owner [num_pages], free list [num_pages], first fresh rank [num_out + 1], and one
// copy (source page, target page, rows) a sequence.
struct Layout {
  int64_t owner, list, base, copies, bytes;
};
__host__ __device__ inline Layout layout_of(int num_pages, int num_out) {
  Layout l;
  l.copies = 0;
  l.owner = 16 * (int64_t)num_out;
  l.list = l.owner + 4 * (int64_t)num_pages;
  l.base = l.list + 4 * (int64_t)num_pages;
  l.bytes = l.base + 4 * ((int64_t)num_out + 1);
  l.bytes = (l.bytes + 15) & ~int64_t(15);
  return l;
}

// What new sequence b continues: its parent's table row, the rows taken over and the rows it
// ends up with. A bad parent or length empties it.
struct Taken {
  const int32_t* row;
  int rows, want;
};
__device__ __forceinline__ Taken taken(const PagesUpdateArgs& a, int b) {
  const int max_rows = a.table_width << a.pv.page_shift;
  const int p = a.parents ? a.parents[b] : b;
  Taken t{nullptr, 0, a.new_lens[b]};
  if (p < -1 || p >= a.num_in || t.want < 0 || t.want > max_rows) {
    record_status(a.status, KVSEL_ERR_BAD_INDEX);
    t.want = 0;
    return t;
  }
  if (p < 0) return t;
  const int len = a.lens[p];
  if (len < 0 || len > max_rows) {
    record_status(a.status, KVSEL_ERR_BAD_INDEX);
    t.want = 0;
    return t;
  }
  t.row = a.table + (int64_t)p * a.table_width;
  t.rows = min(len, t.want);
  return t;
}

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

__global__ void __launch_bounds__(kThreads) pages_table_kernel(const __grid_constant__ PagesUpdateArgs a) {
  __shared__ int warp_sums[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int shift = a.pv.page_shift, mask = a.pv.page_size - 1;
  const Layout lo = layout_of(a.pv.num_pages, a.num_out);
  int* owner = reinterpret_cast<int*>(a.ws + lo.owner);
  int* list = reinterpret_cast<int*>(a.ws + lo.list);
  int* base = reinterpret_cast<int*>(a.ws + lo.base);
  int4* copies = reinterpret_cast<int4*>(a.ws + lo.copies);
  for (int p = tid; p < a.pv.num_pages; p += kThreads) {
    a.ref[p] = 0;
    owner[p] = 0x7fffffff;
  }
  __syncthreads();
  // whole uses, and the lowest user of every started page
  for (int b = warp; b < a.num_out; b += kWarps) {
    const Taken t = taken(a, b);
    for (int i = lane; i < t.rows >> shift; i += 32) {
      const int page = checked_page(a.pv, t.row, i, a.status);
      if (page >= 0) atomicAdd(&a.ref[page], 1);
    }
    if (lane == 0 && (t.rows & mask)) {
      const int page = checked_page(a.pv, t.row, t.rows >> shift, a.status);
      if (page >= 0) atomicMin(&owner[page], b);
    }
  }
  __syncthreads();
  // who keeps its started page; first fresh rank of every sequence
  int demand = 0;
  for (int b0 = 0; b0 < a.num_out; b0 += kThreads) {
    const int b = b0 + tid;
    int fresh = 0;
    if (b < a.num_out) {
      const Taken t = taken(a, b);
      bool keeps = false;
      int src = -1;
      if (t.rows & mask) {
        src = checked_page(a.pv, t.row, t.rows >> shift, a.status);
        keeps = src >= 0 && a.ref[src] == 0 && owner[src] == b;   // only its owner changes it here
        if (keeps) a.ref[src] = 1;
      }
      fresh = ((t.want + mask) >> shift) - (t.rows >> shift) - (keeps ? 1 : 0);
      copies[b] = make_int4(keeps ? -1 : src, -1, t.rows & mask, keeps ? 1 : 0);
    }
    int total;
    const int at = block_prefix(fresh, warp_sums, &total);
    if (b < a.num_out) base[b] = demand + at;
    demand += total;
  }
  // the free pages, ascending
  int nfree = 0;
  for (int p0 = 0; p0 < a.pv.num_pages; p0 += kThreads) {
    const int p = p0 + tid;
    const bool f = p < a.pv.num_pages && a.ref[p] == 0;
    int total;
    const int at = block_prefix(f, warp_sums, &total);
    if (f) list[nfree + at] = p;
    nfree += total;
  }
  __syncthreads();
  if (tid == 0) {
    if (a.free_pages) *a.free_pages = nfree - demand;
    if (demand > nfree) record_status(a.status, KVSEL_ERR_NO_PAGES);
  }
  for (int b = warp; b < a.num_out; b += kWarps) {
    const Taken t = taken(a, b);
    const int4 c = copies[b];
    const int whole = t.rows >> shift, held = whole + c.w, need = (t.want + mask) >> shift;
    int32_t* out = a.table_out + (int64_t)b * a.table_width;
    for (int i = lane; i < a.table_width; i += 32) {
      int page = -1;
      if (i < held) {
        page = checked_page(a.pv, t.row, i, a.status);
      } else if (i < need) {
        const int rank = base[b] + i - held;
        if (rank < nfree) {
          page = list[rank];
          a.ref[page] = 1;
          if (i == whole && c.z) copies[b].y = page;
        }
      }
      out[i] = page;
    }
  }
}

// Rows of started pages for their new holders: one block per (sequence, layer).
__global__ void __launch_bounds__(256) pages_copy_kernel(const __grid_constant__ PagesUpdateArgs a) {
  const Layout lo = layout_of(a.pv.num_pages, a.num_out);
  const int b = blockIdx.x;
  const int4 c = reinterpret_cast<const int4*>(a.ws + lo.copies)[b];
  if (c.x < 0 || c.y < 0) return;
  const int64_t base = (int64_t)blockIdx.y * a.pv.layer_bytes;
  const int64_t so = base + (int64_t)row_units(a.pv, c.x, 0) * kRowUnit;
  const int64_t d0 = base + (int64_t)row_units(a.pv, c.y, 0) * kRowUnit;
  const int64_t vecs = (int64_t)c.z * a.pv.row_units * 2;
  for (int64_t e = threadIdx.x; e < vecs; e += blockDim.x) {
    *reinterpret_cast<uint4*>(a.pv.k + d0 + e * 16) = *reinterpret_cast<const uint4*>(a.pv.k + so + e * 16);
    *reinterpret_cast<uint4*>(a.pv.v + d0 + e * 16) = *reinterpret_cast<const uint4*>(a.pv.v + so + e * 16);
  }
}

}  // namespace

int64_t pages_update_ws(int num_pages, int num_out) { return layout_of(num_pages, num_out).bytes; }

cudaError_t launch_pages_update(const PagesUpdateArgs& a) {
  pages_table_kernel<<<1, kThreads, 0, a.stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e || a.num_out == 0 || a.pv.num_pages == 0) return e;
  pages_copy_kernel<<<dim3((unsigned)a.num_out, (unsigned)a.pv.layers), 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvsel
