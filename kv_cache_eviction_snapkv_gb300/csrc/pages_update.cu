// One step of a page pool's bookkeeping: fork, reorder, grow, cut and free sequences.
//
// New sequence b continues the first m = min(old length, new length) rows of its parent. Its
// columns are: whole pages (column < m / page_size, shared), one started page (m % page_size
// rows), fresh pages up to the new length. Counting the whole uses of every page first makes
// the rest independent of any order: a started page stays with its lowest user if its count
// is 0 and is copied for the others; the pages with count 0 after that are free and go out,
// lowest first, in the order of (sequence, column). A page that is copied from always keeps
// a holder, so it is never handed out in the same step.
//
// Bound by latency: tables of some 100 KB and one count a page, but four dependent passes over
// them. So one cluster of eight blocks makes the tables in one launch, with the cluster's
// hardware barrier between the passes and the blocks' totals in each other's shared memory; a
// second, dependent launch copies the started pages' rows with the whole machine.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace kvsel {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocks = 8;                 // of the cluster
constexpr int kAtOnce = 8;                 // table entries a thread has in flight
constexpr int kTiles = 32;                 // of a page a thread, counted together
constexpr int kPiece = 16384;              // bytes a block copies at a time

// What new sequence b continues: its parent's table row (-1: none), the rows taken over and the
// rows it ends up with.
struct Taken {
  int row, rows, want;
  int fresh_base;            // rank of its first fresh page; the top bit: its started page stays
};

// Workspace: Taken [num_out]; copies (source page, target page, rows) [num_out]; owner [num_pages];
// the blocks' lists of free pages [num_pages]; the number of copies.
struct Layout {
  int64_t copies, owner, list, count, bytes;
};
__host__ __device__ inline Layout layout_of(int num_pages, int num_out) {
  Layout l;
  l.copies = 16 * (int64_t)num_out;
  l.owner = l.copies + 16 * (int64_t)num_out;
  l.list = l.owner + 4 * (int64_t)num_pages;
  l.count = l.list + 4 * (int64_t)num_pages;
  l.bytes = (l.count + 4 + 15) & ~int64_t(15);
  return l;
}

// A bad parent or length empties the sequence.
__device__ __forceinline__ Taken taken(const PagesUpdateArgs& a, int b) {
  const int max_rows = a.table_width << a.pv.page_shift;
  const int p = a.parents ? a.parents[b] : b;
  Taken t{-1, 0, a.new_lens[b], 0};
  const int len = p >= 0 && p < a.num_in ? a.lens[p] : 0;
  if (p < -1 || p >= a.num_in || t.want < 0 || t.want > max_rows || len < 0 || len > max_rows) {
    record_status(a.status, KVSEL_ERR_BAD_INDEX);
    t.want = 0;
  } else if (p >= 0) {
    t.row = p;
    t.rows = min(len, t.want);
  }
  return t;
}

// Exclusive prefix of `v` over the block's threads.
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
  int s = warp_sums[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp ? warp - 1 : 0);
  return (warp ? before : 0) + x - v;
}

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kThreads)
    pages_table_kernel(const __grid_constant__ PagesUpdateArgs a) {
  __shared__ int warp_sums[kWarps], tile_sums[kTiles * kWarps];
  __shared__ int demand_of[kBlocks], free_of[kBlocks];   // every block's, written by their owners
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31;
  const int gtid = rank * kThreads + tid;
  constexpr int kAll = kBlocks * kThreads;
  const int shift = a.pv.page_shift, mask = a.pv.page_size - 1, P = a.pv.num_pages;
  const Layout lo = layout_of(P, a.num_out);
  Taken* const take = reinterpret_cast<Taken*>(a.ws);
  int4* const copies = reinterpret_cast<int4*>(a.ws + lo.copies);
  int* const owner = reinterpret_cast<int*>(a.ws + lo.owner);
  int* const list = reinterpret_cast<int*>(a.ws + lo.list);
  int* const n_copies = reinterpret_cast<int*>(a.ws + lo.count);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  for (int p = gtid; p < P; p += kAll) {
    a.ref[p] = 0;
    owner[p] = 0x7fffffff;
  }
  for (int b = gtid; b < a.num_out; b += kAll) take[b] = taken(a, b);
  if (gtid == 0) *n_copies = 0;
  cluster.sync();

  // whole uses, and the lowest user of every started page
  const uint32_t W = (uint32_t)a.table_width, entries = (uint32_t)a.num_out * W;
  for (uint32_t e0 = gtid; e0 < entries; e0 += kAll * kAtOnce) {
    Taken t[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const uint32_t e = e0 + i * kAll;
      t[i] = take[e < entries ? e / W : 0];
      t[i].want = e < entries ? (int)(e % W) : a.table_width;    // the column
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int whole = t[i].rows >> shift, col = t[i].want;
      if (col > whole || (col == whole && !(t[i].rows & mask))) continue;
      const int page = checked_page(a.pv, a.table + (int64_t)t[i].row * W, col, a.status);
      if (page < 0) continue;
      if (col < whole) atomicAdd(&a.ref[page], 1);
      else atomicMin(&owner[page], (int)((e0 + i * kAll) / W));
    }
  }
  cluster.sync();

  // who keeps its started page; the fresh pages' ranks within this block's run of sequences
  const int b_run = (a.num_out + kBlocks - 1) / kBlocks;
  const int b0 = min(a.num_out, rank * b_run), b1 = min(a.num_out, b0 + b_run);
  int demand = 0;
  for (int bb = b0; bb < b1; bb += kThreads) {
    const int b = bb + tid;
    int fresh = 0;
    Taken t;
    bool keeps = false;
    if (b < b1) {
      t = take[b];
      int src = -1;
      if (t.rows & mask) {
        src = checked_page(a.pv, a.table + (int64_t)t.row * a.table_width, t.rows >> shift, a.status);
        keeps = src >= 0 && a.ref[src] == 0 && owner[src] == b;   // only its owner changes it here
        if (keeps) a.ref[src] = 1;
      }
      fresh = ((t.want + mask) >> shift) - (t.rows >> shift) - (keeps ? 1 : 0);
    }
    int total;
    const int at = block_prefix(fresh, warp_sums, &total);
    if (b < b1) take[b].fresh_base = (demand + at) | (keeps ? (int)0x80000000 : 0);
    demand += total;
  }
  if (tid < kBlocks) *cluster.map_shared_rank(&demand_of[rank], tid) = demand;
  cluster.sync();

  // free pages, ascending: a list for every block's run of pages, no longer than the demand
  int wanted = 0, earlier = 0;
#pragma unroll
  for (int r = 0; r < kBlocks; ++r) {
    wanted += demand_of[r];
    if (r < rank) earlier += demand_of[r];
  }
  const int p_run = (P + kBlocks - 1) / kBlocks;
  const int p0 = (int)min((int64_t)P, (int64_t)rank * p_run), p1 = min(P, p0 + p_run);
  int nfree = 0;
  for (int64_t pp = p0; pp < p1; pp += kTiles * kThreads) {
    const int tiles = (int)min((int64_t)kTiles, (p1 - pp + kThreads - 1) / kThreads);
    uint32_t mine = 0;                   // bit i: page pp + 1024 i + thread is free
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int64_t p = pp + i * kThreads + tid;
      if (p < p1 && a.ref[p] == 0) mine |= 1u << i;
    }
    tile_sums[tid] = 0;
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
      const uint32_t all = __ballot_sync(0xffffffffu, mine >> i & 1u);
      if (lane == 0) tile_sums[i * kWarps + (tid >> 5)] = __popc(all);
    }
    __syncthreads();
    int total;
    const int before = block_prefix(tile_sums[tid], warp_sums, &total);
    tile_sums[tid] = nfree + before;
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
      const uint32_t all = __ballot_sync(0xffffffffu, mine >> i & 1u);
      const int at = tile_sums[i * kWarps + (tid >> 5)] + __popc(all & ((1u << lane) - 1));
      if ((mine >> i & 1u) && at < wanted) list[p0 + at] = (int)(pp + i * kThreads + tid);
    }
    nfree += total;
    __syncthreads();
  }
  if (tid < kBlocks) *cluster.map_shared_rank(&free_of[rank], tid) = nfree;
  cluster.sync();

  int all_free = 0;
#pragma unroll
  for (int r = 0; r < kBlocks; ++r) all_free += free_of[r];
  if (gtid == 0) {
    if (a.free_pages) *a.free_pages = all_free - wanted;
    if (wanted > all_free) record_status(a.status, KVSEL_ERR_NO_PAGES);
  }
  for (uint32_t e0 = gtid; e0 < entries; e0 += kAll * kAtOnce) {
    Taken t[kAtOnce];
    int col[kAtOnce], page[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const uint32_t e = e0 + i * kAll;
      col[i] = e < entries ? (int)(e % W) : -1;
      t[i] = take[col[i] < 0 ? 0 : e / W];
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int held = (t[i].rows >> shift) + (t[i].fresh_base < 0 ? 1 : 0);
      page[i] = -1;
      if (col[i] >= 0 && col[i] < held)
        page[i] = checked_page(a.pv, a.table + (int64_t)t[i].row * W, col[i], a.status);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (col[i] < 0) continue;
      const uint32_t e = e0 + i * kAll;
      const int whole = t[i].rows >> shift, held = whole + (t[i].fresh_base < 0 ? 1 : 0);
      if (col[i] >= held && col[i] < (t[i].want + mask) >> shift) {
        int k = (t[i].fresh_base & 0x7fffffff) + col[i] - held;   // its rank among the free pages
        for (int r = 0; r < (int)(e / W) / b_run; ++r) k += demand_of[r];
        if (k < all_free) {
          int r = 0;
          while (k >= free_of[r]) k -= free_of[r++];
          page[i] = list[(int64_t)r * p_run + k];
          a.ref[page[i]] = 1;
          if (col[i] == whole && (t[i].rows & mask)) {
            const int src = checked_page(a.pv, a.table + (int64_t)t[i].row * W, col[i], a.status);
            if (src >= 0) copies[atomicAdd(n_copies, 1)] = make_int4(src, page[i], t[i].rows & mask, 0);
          }
        }
      }
      a.table_out[e] = page[i];
    }
  }
  cluster.sync();            // no block leaves while another reads its shared memory
}

// Rows of started pages for their new holders, in pieces of kPiece bytes: (copy, layer, K or V,
// piece). The copies' order does not matter: no target is a source or another's target.
__global__ void __launch_bounds__(256) pages_copy_kernel(const __grid_constant__ PagesUpdateArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Layout lo = layout_of(a.pv.num_pages, a.num_out);
  const int n = *reinterpret_cast<const int*>(a.ws + lo.count);
  const int64_t row_bytes = (int64_t)a.pv.row_units * kRowUnit;
  const int pieces = (int)((row_bytes * (a.pv.page_size - 1) + kPiece - 1) / kPiece);
  const int64_t items = (int64_t)n * a.pv.layers * 2 * pieces;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t rest = it / pieces;
    const int64_t from = (it - rest * pieces) * kPiece;
    const int64_t cl = rest >> 1;
    const int layer = (int)(cl % a.pv.layers);
    const int4 c = reinterpret_cast<const int4*>(a.ws + lo.copies)[cl / a.pv.layers];
    const int64_t bytes = min((int64_t)kPiece, c.z * row_bytes - from);
    char* base = (rest & 1 ? a.pv.v : a.pv.k) + layer * a.pv.layer_bytes + from;
    const char* src = base + (int64_t)row_units(a.pv, c.x, 0) * kRowUnit;
    char* dst = base + (int64_t)row_units(a.pv, c.y, 0) * kRowUnit;
    uint4 v[kPiece / 4096];
#pragma unroll
    for (int i = 0; i < kPiece / 4096; ++i) {
      const int e = (i * 256 + threadIdx.x) * 16;
      if (e < bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(src + e));
    }
#pragma unroll
    for (int i = 0; i < kPiece / 4096; ++i) {
      const int e = (i * 256 + threadIdx.x) * 16;
      if (e < bytes) *reinterpret_cast<uint4*>(dst + e) = v[i];
    }
  }
}

}  // namespace

int64_t pages_update_ws(int num_pages, int num_out) { return layout_of(num_pages, num_out).bytes; }

cudaError_t launch_pages_update(const PagesUpdateArgs& a) {
  pages_table_kernel<<<kBlocks, kThreads, 0, a.stream>>>(a);
  cudaError_t e = cudaGetLastError();
  // pages of one row are never started
  if (e || a.num_out == 0 || a.pv.num_pages == 0 || a.pv.page_size == 1) return e;
  cudaLaunchConfig_t cfg{};
  // as many blocks as there can be pieces, or as the SMs hold at a time
  const int64_t pieces = ((int64_t)a.pv.row_units * kRowUnit * (a.pv.page_size - 1) + kPiece - 1) / kPiece;
  const int64_t most = (int64_t)a.num_out * a.pv.layers * 2 * pieces;
  cfg.gridDim = dim3((unsigned)(most < 8 * (int64_t)a.sm_count ? most : 8 * (int64_t)a.sm_count));
  cfg.blockDim = dim3(256);
  cfg.stream = a.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pages_copy_kernel, a);
}

}  // namespace kvsel
