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
// Bound by latency: tables of some 100 KB and two words a page, in dependent passes. A pass
// over global memory costs some two microseconds before its first result and as much to be seen
// by the next, so what the passes exchange stays on chip: a cluster of eight blocks (one block
// where that is enough) holds the pages' counts and lowest users in its shared memory, each
// block a run of pages, and reaches the others' by remote atomics. What follows from a sequence
// alone every block works out for itself. That leaves three barriers: state cleared, uses
// counted, free pages counted; then every free page finds the table entry that it goes to. A
// pool of more pages than the cluster's shared memory holds keeps the two words in memory. A
// second, dependent launch writes the entries that stay and the empty ones, and copies the
// started pages' rows, with the whole machine: eight SMs have few instructions to spare.
//
// Measured: 700 sequences over 150000 pages 19 us (34 us with every entry written by the cluster,
// 240 us by one block), four beams 9.5 us, 224 copies of started pages 39.5 us, 102 MB written.
#include <algorithm>
#include <cooperative_groups.h>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace kvsel {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocks = 8;                 // of the cluster, at most
constexpr int kColumns = 256;              // table columns a warp counts at a time
constexpr int kItems = 3;                  // such pieces that it has in flight
constexpr int kTiles = 4;                  // of a page a thread, numbered together
static_assert(kTiles * kWarps <= kThreads, "a thread a count");
constexpr int kPiece = 32768;              // bytes a block copies at a time
constexpr int kSharedSeqs = 2048;          // sequences whose records fit shared memory
constexpr int kSharedPages = 23 * 1024;    // pages whose state fits a block's shared memory

// What new sequence b continues: its parent's table row (-1: none), the rows taken over, the
// rows it ends up with, and the rank of its first fresh page (~rank if its started page stays
// with it).
struct Taken {
  int row, rows, want, base;
};

// Workspace: copies (source page, target page, rows) [num_out]; the blocks' records of the
// sequences [kBlocks][num_out], the first block's always, for the second launch; lowest users
// [num_pages]; the numbers of copies and of free pages.
struct Layout {
  int64_t taken, owner, count, bytes;
};
__host__ __device__ inline Layout layout_of(int num_pages, int num_out) {
  Layout l;
  l.taken = 16 * (int64_t)num_out;
  l.owner = l.taken + 16 * (int64_t)num_out * kBlocks;
  l.count = (l.owner + 4 * (int64_t)num_pages + 7) & ~int64_t(7);
  l.bytes = (l.count + 8 + 15) & ~int64_t(15);
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

// blocks: of the cluster, the whole grid. shared_pages: whether the pages' state is in shared
// memory, p_run pages a block; run_inverse = ceil(2^40 / p_run) for these.
__global__ void __launch_bounds__(kThreads)
    pages_table_kernel(const __grid_constant__ PagesUpdateArgs a, int blocks, int p_run,
                       uint32_t run_inverse, bool shared_pages) {
  extern __shared__ __align__(16) int smem[];  // counts [p_run], lowest users [p_run]
  __shared__ Taken shared_take[kSharedSeqs];
  __shared__ int warp_sums[kWarps], tile_sums[kTiles * kWarps];
  __shared__ int free_of[kBlocks];       // every block's, written by their owners
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int all = blocks * kThreads, gtid = rank * kThreads + tid;
  const int shift = a.pv.page_shift, mask = a.pv.page_size - 1, P = a.pv.num_pages;
  const Layout lo = layout_of(P, a.num_out);
  int4* const copies = reinterpret_cast<int4*>(a.ws);
  int* const n_copies = reinterpret_cast<int*>(a.ws + lo.count);
  Taken* const take = a.num_out <= kSharedSeqs
                          ? shared_take
                          : reinterpret_cast<Taken*>(a.ws + lo.taken) + (int64_t)rank * a.num_out;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto barrier = [&] {
    if (blocks == 1) __syncthreads();
    else cluster.sync();
  };

  // the pages' state: any block's, and this block's run
  const int p0 = (int)min((int64_t)P, (int64_t)rank * p_run), p1 = (int)min((int64_t)P, (int64_t)p0 + p_run);
  int* const owners = reinterpret_cast<int*>(a.ws + lo.owner);
  int* const own_count = shared_pages ? smem : a.ref + p0;
  int* const own_owner = shared_pages ? smem + p_run : owners + p0;
  auto state_of = [&](int page, int** count, int** owner) {
    if (shared_pages) {
      // page / p_run: exact, as page * p_run < 2^40
      const int r = blocks == 1 ? 0 : (int)((uint64_t)page * run_inverse >> 40), at = page - r * p_run;
      int* s = blocks == 1 ? smem : cluster.map_shared_rank(smem, r);
      *count = s + at;
      *owner = s + p_run + at;
    } else {
      *count = a.ref + page;
      *owner = owners + page;
    }
  };
  if (shared_pages) {
    for (int i = tid; i < p_run / 4; i += kThreads) {
      reinterpret_cast<int4*>(own_count)[i] = make_int4(0, 0, 0, 0);
      reinterpret_cast<int4*>(own_owner)[i] = make_int4(0x7fffffff, 0x7fffffff, 0x7fffffff, 0x7fffffff);
    }
  } else {
    for (int i = tid; i < p1 - p0; i += kThreads) {
      own_count[i] = 0;
      own_owner[i] = 0x7fffffff;
    }
  }
  const int64_t W = a.table_width;
  int started = -1;                      // entry of this thread's first sequence's started page
  for (int b = tid; b < a.num_out; b += kThreads) {
    const Taken t = taken(a, b);
    take[b] = t;
    if (b == tid && (t.rows & mask)) started = __ldg(a.table + t.row * W + (t.rows >> shift));
  }
  if (gtid == 0) *n_copies = 0;
  barrier();

  // whole uses, and the lowest user of every started page
  const uint32_t chunks = (a.table_width + kColumns - 1) / kColumns;
  const uint32_t items = (uint32_t)a.num_out * chunks;           // < 2^31, as num_out * table_width
  constexpr int kCols = kColumns / 32;
  for (uint32_t it0 = gtid >> 5; it0 < items; it0 += all / 32 * kItems) {
    int page[kItems][kCols], b[kItems], c0[kItems], whole[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const uint32_t it = it0 + j * (all / 32);
      const bool in = it < items;
      b[j] = in ? (int)(it / chunks) : 0;
      c0[j] = in ? (int)(it - b[j] * chunks) * kColumns + lane : 0;
      const Taken t = take[b[j]];
      whole[j] = t.rows >> shift;
      const int last = in ? whole[j] + (t.rows & mask ? 1 : 0) : 0;      // columns in use
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        page[j][i] = c0[j] + 32 * i < last ? max(__ldg(a.table + t.row * W + c0[j] + 32 * i), -1) : -2;
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j)
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        if (page[j][i] == -2) continue;
        if (page[j][i] < 0 || page[j][i] >= P) {
          record_status(a.status, KVSEL_ERR_BAD_INDEX);
          continue;
        }
        int *count, *owner;
        state_of(page[j][i], &count, &owner);
        if (c0[j] + 32 * i < whole[j]) atomicAdd(count, 1);
        else atomicMin(owner, b[j]);
      }
  }
  barrier();

  // who keeps its started page; the fresh pages' ranks (in every block alike)
  int wanted = 0;
#pragma unroll 1
  for (int bb = 0; bb < a.num_out; bb += kThreads) {
    const int b = bb + tid;
    int fresh = 0;
    bool keeps = false;
    if (b < a.num_out) {
      const Taken t = take[b];
      if (t.rows & mask) {
        const int src = bb == 0 ? started : __ldg(a.table + t.row * W + (t.rows >> shift));
        if (src >= 0 && src < P) {       // (reported above if not)
          int *count, *owner;
          state_of(src, &count, &owner);
          const int n = *count, lowest = *owner;       // both on their way at once
          keeps = n == 0 && lowest == b;
        }
      }
      fresh = ((t.want + mask) >> shift) - (t.rows >> shift) - (keeps ? 1 : 0);
    }
    int total;
    const int at = wanted + block_prefix(fresh, warp_sums, &total);
    if (b < a.num_out) take[b].base = keeps ? ~at : at;
    wanted += total;
  }

  // A page with a lowest user keeps a holder: that one, or those who hold it whole.
  auto is_free = [&](int64_t p) { return own_count[p - p0] == 0 && own_owner[p - p0] == 0x7fffffff; };
  // This block's first `most` free pages or more, ascending: found(page, its number) for each.
  auto each_free = [&](int most, auto found) {
    int n = 0;
    for (int64_t pp = p0; pp < p1 && n < most; pp += kTiles * kThreads) {
      const int tiles = (int)min((int64_t)kTiles, (p1 - pp + kThreads - 1) / kThreads);
      uint32_t mine = 0;                 // bit i: page pp + 1024 i + thread is free
      for (int i = 0; i < tiles; ++i) {
        const int64_t p = pp + i * kThreads + tid;
        if (p < p1 && is_free(p)) mine |= 1u << i;
      }
      if (tid < kTiles * kWarps) tile_sums[tid] = 0;
      __syncthreads();
      for (int i = 0; i < tiles; ++i) {
        const uint32_t m = __ballot_sync(0xffffffffu, mine >> i & 1u);
        if (lane == 0) tile_sums[i * kWarps + (tid >> 5)] = __popc(m);
      }
      __syncthreads();
      int total;
      const int at = n + block_prefix(tid < kTiles * kWarps ? tile_sums[tid] : 0, warp_sums, &total);
      if (tid < kTiles * kWarps) tile_sums[tid] = at;
      __syncthreads();
      for (int i = 0; i < tiles; ++i) {
        const uint32_t m = __ballot_sync(0xffffffffu, mine >> i & 1u);
        if (mine >> i & 1u)
          found((int)(pp + i * kThreads + tid),
                tile_sums[i * kWarps + (tid >> 5)] + __popc(m & ((1u << lane) - 1)));
      }
      n += total;
      __syncthreads();
    }
  };
  // Free pages of this block's run, and the held pages' references (the free ones get theirs as
  // they are handed out). In memory the counts are the references already, but for the started
  // pages', which other blocks may still be reading.
  int nfree;
  {
    int n = 0;
    if (shared_pages && (reinterpret_cast<uintptr_t>(a.ref) & 15) == 0) {
      const int end = p1 - p0;           // p0 is a multiple of 4
      for (int i = 4 * tid; i < end; i += 4 * kThreads) {
        const int4 c = *reinterpret_cast<const int4*>(own_count + i);
        const int4 o = *reinterpret_cast<const int4*>(own_owner + i);
        const int4 r = make_int4(c.x ? c.x : o.x != 0x7fffffff, c.y ? c.y : o.y != 0x7fffffff,
                                 c.z ? c.z : o.z != 0x7fffffff, c.w ? c.w : o.w != 0x7fffffff);
        if (i + 4 <= end) {
          n += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
          *reinterpret_cast<int4*>(a.ref + p0 + i) = r;
        } else {
          const int left[3] = {r.x, r.y, r.z};
#pragma unroll
          for (int k = 0; k < 3; ++k)
            if (i + k < end) {
              n += left[k] == 0;
              a.ref[p0 + i + k] = left[k];
            }
        }
      }
    } else if (shared_pages) {
      for (int i = tid; i < p1 - p0; i += kThreads) {
        const int c = own_count[i];
        const bool started = own_owner[i] != 0x7fffffff;
        n += c == 0 && !started;
        a.ref[p0 + i] = c ? c : started;
      }
    } else {
      for (int p = p0 + tid; p < p1; p += kThreads) n += is_free(p);
    }
    block_prefix(n, warp_sums, &nfree);
  }
  if (blocks == 1) {
    if (tid == 0) free_of[0] = nfree;
  } else if (tid < blocks) {
    cluster.map_shared_rank(free_of, tid)[rank] = nfree;
  }
  barrier();

  int all_free = 0, before = 0;
  for (int r = 0; r < blocks; ++r) {
    if (r < rank) before += free_of[r];
    all_free += free_of[r];
  }
  if (gtid == 0) {
    n_copies[1] = all_free;
    if (a.free_pages) *a.free_pages = all_free - wanted;
    if (wanted > all_free) record_status(a.status, KVSEL_ERR_NO_PAGES);
  }
  if (!shared_pages)
    for (int i = tid; i < p1 - p0; i += kThreads)
      if (own_count[i] == 0 && own_owner[i] != 0x7fffffff) own_count[i] = 1;
  __syncthreads();
  if (before < wanted) {
    each_free(wanted - before, [&](int page, int k) {
      k += before;
      if (k >= wanted) return;
      auto base_of = [&](int b) { return take[b].base < 0 ? ~take[b].base : take[b].base; };
      const int b = upper_find(a.num_out, k, base_of);
      const Taken t = take[b];
      const int whole = t.rows >> shift, col = whole + (t.base < 0 ? 1 : 0) + k - base_of(b);
      a.table_out[b * W + col] = page;
      a.ref[page] = 1;
      if (col == whole && (t.rows & mask)) {
        const int src = checked_page(a.pv, a.table + t.row * W, col, a.status);
        if (src >= 0) copies[atomicAdd(n_copies, 1)] = make_int4(src, page, t.rows & mask, 0);
      }
    });
  }
  if (rank == 0 && take == shared_take)
    for (int b = tid; b < a.num_out; b += kThreads)
      reinterpret_cast<Taken*>(a.ws + lo.taken)[b] = take[b];
}

// The table entries that are held, and the empty ones (the fresh ones are there).
__device__ __forceinline__ void other_entries(const PagesUpdateArgs& a, const Layout& lo, int all_free) {
  const int shift = a.pv.page_shift, mask = a.pv.page_size - 1;
  const Taken* take = reinterpret_cast<const Taken*>(a.ws + lo.taken);
  const int64_t W = a.table_width;
  const uint32_t entries = (uint32_t)(a.num_out * W);        // < 2^31
  for (uint32_t e = blockIdx.x * blockDim.x + threadIdx.x; e < entries; e += gridDim.x * blockDim.x) {
    const int b = (int)(e / (uint32_t)W), col = (int)(e - b * (uint32_t)W);
    const Taken t = take[b];
    const int held = (t.rows >> shift) + (t.base < 0 ? 1 : 0);
    int page = -1;
    if (col < held)
      page = checked_page(a.pv, a.table + t.row * W, col, a.status);
    else if (col < (t.want + mask) >> shift && (t.base < 0 ? ~t.base : t.base) + col - held < all_free)
      continue;
    a.table_out[e] = page;
  }
}

// Rows of started pages for their new holders, in pieces of kPiece bytes: (copy, layer, K or V,
// piece). The copies' order does not matter: no target is a source or another's target.
__global__ void __launch_bounds__(256, 3) pages_copy_kernel(const __grid_constant__ PagesUpdateArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Layout lo = layout_of(a.pv.num_pages, a.num_out);
  const int2 counts = *reinterpret_cast<const int2*>(a.ws + lo.count);
  const int n = counts.x;
  other_entries(a, lo, counts.y);
  const int64_t row_bytes = (int64_t)a.pv.row_units * kRowUnit;
  const int pieces = (int)((row_bytes * (a.pv.page_size - 1) + kPiece - 1) / kPiece);
  const int64_t items = (int64_t)n * a.pv.layers * 2 * pieces;
  struct Piece {
    char* src;
    char* dst;
    int bytes;
  };
  auto piece = [&](int64_t it) {
    Piece x{nullptr, nullptr, 0};
    if (it >= items) return x;
    const int64_t rest = quotient(it, pieces);
    const int64_t from = (it - rest * pieces) * kPiece;
    const int64_t cl = rest >> 1, at = quotient(cl, a.pv.layers);
    const int layer = (int)(cl - at * a.pv.layers);
    const int4 c = reinterpret_cast<const int4*>(a.ws)[at];
    char* base = (rest & 1 ? a.pv.v : a.pv.k) + layer * a.pv.layer_bytes + from;
    x.src = base + (int64_t)row_units(a.pv, c.x, 0) * kRowUnit;
    x.dst = base + (int64_t)row_units(a.pv, c.y, 0) * kRowUnit;
    x.bytes = (int)max((int64_t)0, min((int64_t)kPiece, c.z * row_bytes - from));
    return x;
  };
  Piece next = piece(blockIdx.x);
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const Piece x = next;
    uint4 v[kPiece / 4096];
#pragma unroll
    for (int i = 0; i < kPiece / 4096; ++i) {
      const int e = (i * 256 + threadIdx.x) * 16;
      if (e < x.bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(x.src + e));
    }
    next = piece(it + gridDim.x);          // while this one's rows arrive
#pragma unroll
    for (int i = 0; i < kPiece / 4096; ++i) {
      const int e = (i * 256 + threadIdx.x) * 16;
      if (e < x.bytes) *reinterpret_cast<uint4*>(x.dst + e) = v[i];
    }
  }
}

}  // namespace

int64_t pages_update_ws(int num_pages, int num_out) { return layout_of(num_pages, num_out).bytes; }

cudaError_t launch_pages_update(const PagesUpdateArgs& a) {
  // One block where it has few pages and columns to count: its barriers are much cheaper (four
  // beams 10.3 us, 14 in the cluster; 256 samples of 25 pages 48.7, 44.2 in the cluster). A pool
  // that the blocks' shared memory does not hold takes eight and global memory.
  const int64_t items = (int64_t)a.num_out * ((a.table_width + kColumns - 1) / kColumns);
  const bool one = a.pv.num_pages <= kSharedPages / 4 && items <= 4 * kWarps;
  const int blocks = one ? 1 : kBlocks;
  const int p_run = (int)std::max<int64_t>((((int64_t)a.pv.num_pages + blocks - 1) / blocks + 3) & ~int64_t(3), 1024);
  const bool shared_pages = p_run <= kSharedPages;
  const uint32_t run_inverse = (uint32_t)(((uint64_t(1) << 40) + p_run - 1) / p_run);
  static_assert(kSharedPages * 8 + kSharedSeqs * 16 + 8 * 1024 <= 227 * 1024, "fits shared memory");
  // always the same value: another thread's call may come between
  cudaError_t e = cudaFuncSetAttribute(pages_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSharedPages * 8);
  if (e) return e;
  {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = shared_pages ? (size_t)p_run * 8 : 0;
    cfg.stream = a.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, pages_table_kernel, a, blocks, p_run, run_inverse, shared_pages)))
      return e;
  }
  if (a.num_out == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  // as many blocks as there can be pieces or entries for, or some five times what the SMs hold at a
  // time: shares of a few pieces even out (three blocks an SM 44.8 us for eight samples, eight
  // 40.8, sixteen 39.5, one a piece 42.5). (Pages of one row are never started.)
  const int64_t pieces = ((int64_t)a.pv.row_units * kRowUnit * (a.pv.page_size - 1) + kPiece - 1) / kPiece;
  const int64_t most = std::max((int64_t)a.num_out * a.pv.layers * 2 * pieces,
                                ((int64_t)a.num_out * a.table_width + 255) / 256);
  cfg.gridDim = dim3((unsigned)std::min(most, 16 * (int64_t)a.sm_count));
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
