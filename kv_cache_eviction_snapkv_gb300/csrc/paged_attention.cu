// One new query per (layer, sequence, query head) over a paged cache.
//
// Mathematics: s_j = q . k_j / sqrt(D) over the rows j < len, running maximum m and sum l of
// exp(s - m), out = sum_j exp(s_j - m) v_j / l, lse = m + ln l; an empty sequence has out = 0
// and lse = -inf. Base-2 units until the end.
//
// Bound by memory: every K and V row is read once for all the query heads that share it, so
// the products are small matrix products, S^T = K Q^T (16 rows x 8 heads a step) and
// O^T = V^T P^T, which fit mma.sync's m16n8 tile as they are: rows or dimensions are the 16,
// a group's heads the 8. (tcgen05 wants 128 rows and a trip through tensor memory for P; the
// products take a few percent of the time a step's bytes take to arrive.) Both operands come
// straight from global memory to registers: a dot product may take its dimensions in any
// order, so a lane's 32-byte pieces of K rows serve as the fragments, with q loaded in the same
// order; V's fragments pair two rows' values, which a byte permutation makes of two rows'
// pieces. No shared memory, no barrier in the loop; the next step's K loads go out when
// this step's K is used up, V's likewise, so a warp has about a step's bytes in flight all the
// time.
//
// Split: all (layer, sequence, head) instances' row blocks form one line, which the blocks of
// one wave cut into equal pieces, from the lengths on the device: a batch of any mix of lengths
// takes every SM the same time, and a single long sequence uses them all. A piece that holds an
// instance whole writes its result; the others write a partial (max, sum, weighted values) to
// one of two slots a block has, and a second, dependent launch joins them in order (the same
// bits every time).
#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

// What the launch fixes; the rest follows from the lengths.
struct AttnGeom {
  int G;              // query heads per cache head
  int wk_shift;       // log2 of the warps that split the rows (the others split the heads)
  int heads;          // query heads a block takes
  int HG;             // head groups: ceil(G / heads)
  int grid;
};

// Workspace: what each block's split instance is, then the partials [grid][2][heads]: base-2
// max and sum, and the weighted values [D].
struct SplitInfo {
  int64_t first_head; // index of its first query head in out / D, -1: no instance to join
  int last;           // last block that has a piece of it
  int heads;
};
__host__ __device__ inline int64_t ws_ml(int grid) { return 16 * (int64_t)grid; }
__host__ __device__ inline int64_t ws_acc(int grid, int heads) {
  return ws_ml(grid) + ((16 * (int64_t)grid * heads + 15) & ~int64_t(15));
}

template <int N>
struct Bytes {
  uint32_t r[N / 4];
};

__device__ __forceinline__ void load_piece(Bytes<32>& b, const char* p) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(b.r[0]), "=r"(b.r[1]), "=r"(b.r[2]), "=r"(b.r[3]), "=r"(b.r[4]), "=r"(b.r[5]),
                 "=r"(b.r[6]), "=r"(b.r[7])
               : "l"(p));
}
__device__ __forceinline__ void load_piece(Bytes<16>& b, const char* p) {
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(b.r[0]), "=r"(b.r[1]), "=r"(b.r[2]), "=r"(b.r[3])
               : "l"(p));
}
template <int N>
__device__ __forceinline__ void load_row_piece(uint32_t (&dst)[N], const char* p, int step) {
  constexpr int kB = N * 4 >= 32 ? 32 : 16;
#pragma unroll
  for (int c = 0; c < N * 4 / kB; ++c) {
    Bytes<kB> b;
    load_piece(b, p + c * step);
#pragma unroll
    for (int i = 0; i < kB / 4; ++i) dst[c * (kB / 4) + i] = b.r[i];
  }
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two floats to bf16, `a` in the lower half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t y;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(b), "f"(a));
  return y;
}
// x = hi + lo in two tf32 values: 22 bits of x.
__device__ __forceinline__ void split_tf32(float x, uint32_t* hi, uint32_t* lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(*hi) : "f"(x));
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(*lo) : "f"(x - __uint_as_float(*hi)));
}

// A warp's part of a step: 16 rows x 8 * NT heads. Lane (g, t) = (lane / 4, lane % 4) holds of
// S^T rows g and g + 8, heads 2t and 2t + 1; of O^T (m-tile i) dimensions g * D/8 + 2i and
// + 1, heads 2t and 2t + 1. kr, vr: its pieces of K rows g, g + 8 and of V rows 2t, 2t + 1,
// 2t + 8, 2t + 9.
template <typename T, int D, int NT>
struct Step {
  static constexpr int kEb = sizeof(T);
  static constexpr int kKw = D * kEb / 16;            // words of a K row a lane holds
  static constexpr int kVw = D * kEb / 32;            // words of a V row a lane holds
  static constexpr int kMt = D / 16;                  // m-tiles of O^T
  static constexpr int kQ = kEb == 2 ? kKw * NT : 1;  // q fragments in registers (bf16)
  uint32_t kr[2][kKw];
  uint32_t vr[4][kVw];
  uint32_t qf[kQ];
  float o[NT][kMt][4];
  float m[NT][2], l[NT][2];

  __device__ __forceinline__ void load_k(const char* base, uint32_t off, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t o32 = __shfl_sync(0xffffffffu, off, g + 8 * i);
      load_row_piece(kr[i], base + (int64_t)o32 * kRowUnit + t * 32, 128);
    }
  }
  __device__ __forceinline__ void load_v(const char* base, uint32_t off, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t o32 = __shfl_sync(0xffffffffu, off, 2 * t + (i & 1) + 8 * (i >> 1));
      load_row_piece(vr[i], base + (int64_t)o32 * kRowUnit + g * (kVw * 4), 32);
    }
  }
  // S^T of this step's rows and heads. qs: fp32's split q fragments in shared memory.
  __device__ __forceinline__ void scores(float (&s)[NT][4], const uint4* qs, int lane) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float acc[2][4] = {};
      if constexpr (kEb == 2) {
#pragma unroll
        for (int k = 0; k < kKw / 2; ++k)
          mma_bf16(acc[k & 1], kr[0][2 * k], kr[1][2 * k], kr[0][2 * k + 1], kr[1][2 * k + 1],
                   qf[n * kKw + 2 * k], qf[n * kKw + 2 * k + 1]);
      } else {
#pragma unroll
        for (int k = 0; k < kKw / 2; ++k) {
          const uint4 b = qs[(n * (kKw / 2) + k) * 32 + lane];   // hi, hi, lo, lo
          uint32_t h[4], w[4];
          split_tf32(__uint_as_float(kr[0][2 * k]), &h[0], &w[0]);
          split_tf32(__uint_as_float(kr[1][2 * k]), &h[1], &w[1]);
          split_tf32(__uint_as_float(kr[0][2 * k + 1]), &h[2], &w[2]);
          split_tf32(__uint_as_float(kr[1][2 * k + 1]), &h[3], &w[3]);
          mma_tf32(acc[0], h[0], h[1], h[2], h[3], b.x, b.y);
          mma_tf32(acc[1], w[0], w[1], w[2], w[3], b.x, b.y);
          mma_tf32(acc[1], h[0], h[1], h[2], h[3], b.z, b.w);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = acc[0][i] + acc[1][i];
    }
  }
  // O^T += V^T P^T; p: this lane's weights, in S^T's places.
  __device__ __forceinline__ void values(const float (&p)[NT][4]) {
    if constexpr (kEb == 2) {
      // weights as a sum of two bf16 (2^-17 of the weight): one would cost 2^-9
      uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = p[n][2 * i], p1 = p[n][2 * i + 1];
          const uint32_t hi = pack_bf16(p0, p1);
          const uint32_t lo = pack_bf16(p0 - __uint_as_float(hi << 16),
                                        p1 - __uint_as_float(hi & 0xffff0000u));
          bh[n][i] = transposed(hi);
          bl[n][i] = transposed(lo);
        }
#pragma unroll
      for (int i = 0; i < kMt; ++i) {
        const uint32_t a0 = __byte_perm(vr[0][i], vr[1][i], 0x5410);
        const uint32_t a1 = __byte_perm(vr[0][i], vr[1][i], 0x7632);
        const uint32_t a2 = __byte_perm(vr[2][i], vr[3][i], 0x5410);
        const uint32_t a3 = __byte_perm(vr[2][i], vr[3][i], 0x7632);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_bf16(o[n][i], a0, a1, a2, a3, bh[n][0], bh[n][1]);
          mma_bf16(o[n][i], a0, a1, a2, a3, bl[n][0], bl[n][1]);
        }
      }
    } else {
      uint32_t ph[NT][4], pl[NT][4];               // rows 2t, 2t + 1, 2t + 8, 2t + 9 of head g
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = __float_as_uint(p[n][2 * i]), y = __float_as_uint(p[n][2 * i + 1]);
          const uint32_t top = transposed(__byte_perm(x, y, 0x7632));
          const uint32_t low = transposed(__byte_perm(x, y, 0x5410));
          split_tf32(__uint_as_float(__byte_perm(low, top, 0x5410)), &ph[n][2 * i], &pl[n][2 * i]);
          split_tf32(__uint_as_float(__byte_perm(low, top, 0x7632)), &ph[n][2 * i + 1],
                     &pl[n][2 * i + 1]);
        }
#pragma unroll
      for (int i = 0; i < kMt; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h[4], w[4];
          split_tf32(__uint_as_float(vr[2 * k][2 * i]), &h[0], &w[0]);
          split_tf32(__uint_as_float(vr[2 * k][2 * i + 1]), &h[1], &w[1]);
          split_tf32(__uint_as_float(vr[2 * k + 1][2 * i]), &h[2], &w[2]);
          split_tf32(__uint_as_float(vr[2 * k + 1][2 * i + 1]), &h[3], &w[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_tf32(o[n][i], h[0], h[1], h[2], h[3], ph[n][2 * k], ph[n][2 * k + 1]);
            mma_tf32(o[n][i], w[0], w[1], w[2], w[3], ph[n][2 * k], ph[n][2 * k + 1]);
            mma_tf32(o[n][i], h[0], h[1], h[2], h[3], pl[n][2 * k], pl[n][2 * k + 1]);
          }
        }
    }
  }
};

// Offsets of 16 rows from j0 on, lane i (mod 16) that of row j0 + i; `valid`: which rows count.
// Rows that do not count get the offset of one that does.
__device__ __forceinline__ uint32_t row_offsets(const PagedView& pv, const int32_t* trow, int j0,
                                                int len, uint32_t* valid, int* status) {
  const int lane = threadIdx.x & 31, j = j0 + (lane & 15);
  uint32_t off = 0;
  int page = -1;
  if (j < len) {
    page = checked_page(pv, trow, j >> pv.page_shift, status);
    off = row_units(pv, max(page, 0), j & (pv.page_size - 1));
  }
  const uint32_t v = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
  *valid = v;
  const uint32_t other = __shfl_sync(0xffffffffu, off, v ? __ffs(v) - 1 : 0);
  return page >= 0 ? off : other;
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && NT == 1 ? 3 : 2)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ AttnGeom gm) {
  using St = Step<T, D, NT>;
  constexpr int kHw = 8 * NT;                     // heads of a warp
  constexpr int kRow = D + 4;                     // padded rows of the joined values
  extern __shared__ int pre[];                    // row blocks before sequence b
  __shared__ int warp_sums[kWarps];
  __shared__ float wm[kWarps][kHw], wl[kWarps][kHw];
  // a warp's own part: fp32's split q fragments while it walks its rows, its values after that
  constexpr int kQs = sizeof(T) == 4 ? NT * (D / 8) * 32 : 0;
  constexpr int kOwn = kQs * 16 > kHw * kRow * 4 ? kQs * 16 : kHw * kRow * 4;
  __shared__ __align__(16) unsigned char own[kWarps][kOwn];
  auto wo = [&](int w, int h) { return reinterpret_cast<float*>(own[w]) + h * kRow; };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // row blocks before every sequence
  const int wk = 1 << gm.wk_shift, block_shift = 4 + gm.wk_shift;
  const int max_rows = a.table_width << a.pv.page_shift;
  int nb = 0;
  for (int b0 = 0; b0 < a.S; b0 += kThreads) {
    const int b = b0 + tid;
    int x = 0;
    if (b < a.S)
      x = (int)(((int64_t)checked_len(a.lens[b], max_rows, a.status) + (1 << block_shift) - 1) >> block_shift);
    int y = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, off);
      if (lane >= off) y += z;
    }
    if (lane == 31) warp_sums[warp] = y;
    __syncthreads();
    int before = nb, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sums[w];
      all += warp_sums[w];
    }
    if (b < a.S) pre[b] = before + y - x;
    nb += all;
    __syncthreads();
  }
  if (tid == 0) pre[a.S] = nb;
  __syncthreads();

  const int HH = a.pv.Hkv * gm.HG;
  const int64_t per_layer = (int64_t)nb * HH;
  const int64_t units = per_layer * a.pv.layers;
  const int parts = (int)min((int64_t)gm.grid, units);       // every part has a row block at least
  auto part_start = [&](int64_t c) { return c * units / parts; };
  const bool works = (int)blockIdx.x < parts;
  const int64_t u0 = works ? part_start(blockIdx.x) : 0, u1 = works ? part_start(blockIdx.x + 1) : 0;

  // empty sequences
  for (int b = blockIdx.x; b < a.S; b += gm.grid) {
    if (pre[b + 1] != pre[b]) continue;
    for (int layer = 0; layer < a.pv.layers; ++layer) {
      const int64_t at = ((int64_t)layer * a.S + b) * a.H;
      for (int i = tid; i < a.H * D; i += kThreads) a.out[at * D + i] = 0.f;
      if (a.lse)
        for (int i = tid; i < a.H; i += kThreads) a.lse[at + i] = -INFINITY;
    }
  }

  SplitInfo info{-1, 0, 0};
  float* ml = reinterpret_cast<float*>(a.ws + ws_ml(gm.grid));
  float* acc = reinterpret_cast<float*>(a.ws + ws_acc(gm.grid, gm.heads));
  const int wh = warp >> gm.wk_shift, wrow = (warp & (wk - 1)) * 16;

  for (int64_t u = u0; u < u1;) {
    const int layer = (int)(u / per_layer);
    const int64_t rem = u - layer * per_layer;
    const int b = upper_find(a.S, (int)(rem / HH), [&](int i) { return pre[i]; });
    const int n_blk = pre[b + 1] - pre[b];
    const int64_t local = rem - (int64_t)pre[b] * HH;
    const int head = (int)(local / n_blk), blk0 = (int)(local - (int64_t)head * n_blk);
    const int n = (int)min((int64_t)(n_blk - blk0), u1 - u);
    const int kvh = head / gm.HG, hg = head - kvh * gm.HG;
    const int n_heads = min(gm.heads, gm.G - hg * gm.heads);
    const int64_t first_head = ((int64_t)layer * a.S + b) * a.H + kvh * gm.G + hg * gm.heads;
    const int len = min(max(a.lens[b], 0), max_rows);
    const int32_t* trow = a.table + (int64_t)b * a.table_width;
    const int64_t base = layer * a.pv.layer_bytes + (int64_t)kvh * a.pv.head_units * kRowUnit;
    const char* kb = a.pv.k + base;
    const char* vb = a.pv.v + base;

    St st;
    // q in the order of K's pieces; heads past the group's are zero
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      const int h = wh * kHw + x * 8 + g;
      uint32_t w[St::kKw] = {};
      if (h < n_heads)
        load_row_piece(w, static_cast<const char*>(a.q) + (first_head + h) * (D * St::kEb) + t * 32, 128);
      if constexpr (St::kEb == 2) {
#pragma unroll
        for (int i = 0; i < St::kKw; ++i) st.qf[x * St::kKw + i] = w[i];
      } else {
#pragma unroll
        for (int i = 0; i < St::kKw / 2; ++i) {
          uint4 f;
          split_tf32(__uint_as_float(w[2 * i]), &f.x, &f.z);
          split_tf32(__uint_as_float(w[2 * i + 1]), &f.y, &f.w);
          reinterpret_cast<uint4*>(own[warp])[(x * (St::kKw / 2) + i) * 32 + lane] = f;
        }
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < St::kMt; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) st.o[x][i][k] = 0.f;
      st.m[x][0] = st.m[x][1] = -INFINITY;
      st.l[x][0] = st.l[x][1] = 0.f;
    }

    const uint4* qs = reinterpret_cast<const uint4*>(own[warp]);
    int j = (blk0 << block_shift) + wrow;
    const int j_end = min(len, (blk0 + n) << block_shift);
    uint32_t valid = 0, next_valid = 0;
    uint32_t off = 0, next = 0;
    if (j < j_end) {
      off = row_offsets(a.pv, trow, j, len, &valid, a.status);
      if (valid) {
        st.load_k(kb, off, lane);
        st.load_v(vb, off, lane);
      }
    }
    while (j < j_end) {
      const int jn = j + (wk << 4);
      next_valid = 0;
      if (jn < j_end) next = row_offsets(a.pv, trow, jn, len, &next_valid, a.status);
      float s[NT][4];
      if (valid) {
        st.scores(s, qs, lane);
        if (next_valid) st.load_k(kb, next, lane);
        const bool ok0 = valid >> g & 1u, ok1 = valid >> (g + 8) & 1u;
        bool moved = false;
        float f[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            s[x][c] = ok0 ? s[x][c] * a.scale_log2 : -INFINITY;
            s[x][2 + c] = ok1 ? s[x][2 + c] * a.scale_log2 : -INFINITY;
            float mx = fmaxf(s[x][c], s[x][2 + c]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            mx = fmaxf(mx, st.m[x][c]);
            const float ref = mx == -INFINITY ? 0.f : mx;
            f[x][c] = ex2(st.m[x][c] - ref);
            moved |= mx != st.m[x][c];
            st.m[x][c] = mx;
            // -inf gives 0; NaN (and +inf, whose maximum it is) gives NaN
            s[x][c] = ex2(s[x][c] - ref);
            s[x][2 + c] = ex2(s[x][2 + c] - ref);
          }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            st.l[x][0] *= f[x][0];
            st.l[x][1] *= f[x][1];
#pragma unroll
            for (int i = 0; i < St::kMt; ++i) {
              st.o[x][i][0] *= f[x][0];
              st.o[x][i][1] *= f[x][1];
              st.o[x][i][2] *= f[x][0];
              st.o[x][i][3] *= f[x][1];
            }
          }
        }
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          st.l[x][0] += s[x][0] + s[x][2];
          st.l[x][1] += s[x][1] + s[x][3];
        }
        st.values(s);
      } else if (next_valid) {
        st.load_k(kb, next, lane);
      }
      if (next_valid) st.load_v(vb, next, lane);
      off = next;
      valid = next_valid;
      j = jn;
    }

    // the warps' results, joined through shared memory
    __syncwarp();
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = st.l[x][c];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) {
          wm[warp][x * 8 + 2 * t + c] = st.m[x][c];
          wl[warp][x * 8 + 2 * t + c] = l;
        }
        float* w = wo(warp, x * 8 + 2 * t + c) + g * (D / 8);
#pragma unroll
        for (int i = 0; i < St::kMt; i += 2)
          *reinterpret_cast<float4*>(w + 2 * i) =
              make_float4(st.o[x][i][c], st.o[x][i][2 + c], st.o[x][i + 1][c], st.o[x][i + 1][2 + c]);
      }
    }
    __syncthreads();
    const bool whole = blk0 == 0 && n == n_blk;
    const int slot = blk0 > 0 ? 0 : 1;
    bool bad = false;
    for (int e = tid; e < n_heads * (D / 4); e += kThreads) {
      const int h = e / (D / 4), d = e - h * (D / 4);
      const int w0 = (h / kHw) << gm.wk_shift, hw = h % kHw;
      float mx = -INFINITY;
      for (int w = 0; w < wk; ++w) mx = fmaxf(mx, wm[w0 + w][hw]);
      float sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < wk; ++w) {
        const float m = wm[w0 + w][hw];
        const float f = m == -INFINITY ? 0.f : ex2(m - mx);   // a NaN sum stays NaN
        sum = fmaf(wl[w0 + w][hw], f, sum);
        const float4 y = *reinterpret_cast<const float4*>(wo(w0 + w, hw) + 4 * d);
        v.x = fmaf(y.x, f, v.x);
        v.y = fmaf(y.y, f, v.y);
        v.z = fmaf(y.z, f, v.z);
        v.w = fmaf(y.w, f, v.w);
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        bad |= !finite_f(sum) || !finite_f(v.x) || !finite_f(v.y) || !finite_f(v.z) || !finite_f(v.w);
        reinterpret_cast<float4*>(a.out + (first_head + h) * D)[d] = v;
        if (d == 0 && a.lse)
          a.lse[first_head + h] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
      } else {
        const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * gm.heads + h;
        reinterpret_cast<float4*>(acc + at * D)[d] = v;
        if (d == 0) reinterpret_cast<float2*>(ml)[at] = make_float2(mx, sum);
      }
    }
    if (bad) record_status(a.status, KVSEL_ERR_NONFINITE);
    if (blk0 == 0 && !whole) {
      // its last piece is the last part's that starts before its end
      const int64_t end = u + n_blk;
      info.first_head = first_head;
      info.heads = n_heads;
      info.last = (int)(end * parts / units);
      if (info.last >= parts) info.last = parts - 1;
      while (part_start(info.last) >= end) --info.last;
      while (info.last + 1 < parts && part_start(info.last + 1) < end) ++info.last;
    }
    __syncthreads();
    u += n;
  }
  if (tid == 0) reinterpret_cast<SplitInfo*>(a.ws)[blockIdx.x] = info;
}

// Joins the pieces of block x's split instance, head y: slot 1 of block x, then slot 0 of the
// blocks up to `last`.
template <int D>
__global__ void __launch_bounds__(D) paged_join_kernel(const __grid_constant__ PagedAttnArgs a,
                                                       const __grid_constant__ AttnGeom gm) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x = blockIdx.x, h = blockIdx.y, d = threadIdx.x;
  const SplitInfo info = reinterpret_cast<const SplitInfo*>(a.ws)[x];
  if (info.first_head < 0 || h >= info.heads) return;
  const float2* ml = reinterpret_cast<const float2*>(a.ws + ws_ml(gm.grid));
  const float* acc = reinterpret_cast<const float*>(a.ws + ws_acc(gm.grid, gm.heads));
  auto at = [&](int c) { return ((int64_t)c * 2 + (c == x ? 1 : 0)) * gm.heads + h; };
  float mx = -INFINITY;
  for (int c = x; c <= info.last; ++c) mx = fmaxf(mx, ml[at(c)].x);
  float sum = 0.f, v = 0.f;
#pragma unroll 4
  for (int c = x; c <= info.last; ++c) {
    const float2 y = ml[at(c)];
    const float f = y.x == -INFINITY ? 0.f : ex2(y.x - mx);
    sum = fmaf(y.y, f, sum);
    v = fmaf(acc[at(c) * D + d], f, v);
  }
  v = sum == 0.f ? 0.f : v / sum;
  a.out[(info.first_head + h) * D + d] = v;
  if (d == 0 && a.lse)
    a.lse[info.first_head + h] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
  if (!finite_f(sum) || !finite_f(v)) record_status(a.status, KVSEL_ERR_NONFINITE);
}

// Heads per warp: 8, or 16 in bf16 once a group has more (its fragments of V then serve two
// products; fp32's registers do not hold them). Warps beyond the group's heads split the rows.
int head_tiles(const PagedView& pv, int G) { return pv.dtype == KVSEL_BF16 && G > 8 ? 2 : 1; }

AttnGeom geometry(const PagedView& pv, int H, int sm_count) {
  AttnGeom gm;
  gm.G = H / pv.Hkv;
  const int nt = head_tiles(pv, gm.G);
  int wh = 1;
  while (wh < kWarps && wh * 8 * nt < gm.G) wh *= 2;
  gm.wk_shift = wh == 1 ? 2 : wh == 2 ? 1 : 0;
  gm.heads = gm.G < wh * 8 * nt ? gm.G : wh * 8 * nt;
  gm.HG = (gm.G + gm.heads - 1) / gm.heads;
  // one wave: three blocks an SM with 8 bf16 heads a warp, else two (registers)
  gm.grid = sm_count * (pv.dtype == KVSEL_BF16 && nt == 1 ? 3 : 2);
  return gm;
}

template <typename T, int D, int NT>
cudaError_t launch(const PagedAttnArgs& a, const AttnGeom& gm) {
  const int smem = (a.S + 1) * (int)sizeof(int);
  cudaError_t e;
  // with the static part, at most 67 KB: two or three blocks still share an SM. (Always the
  // same value: another thread's call may come between.)
  if (smem > 8 * 1024 &&
      (e = cudaFuncSetAttribute(paged_attn_kernel<T, D, NT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (kMaxPagedSeqs + 1) * (int)sizeof(int))))
    return e;
  paged_attn_kernel<T, D, NT><<<gm.grid, kThreads, smem, a.stream>>>(a, gm);
  e = cudaGetLastError();
  if (e) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)gm.grid, (unsigned)gm.heads);
  cfg.blockDim = dim3(D);
  cfg.stream = a.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, a, gm);
}

}  // namespace

int64_t paged_attention_ws(const PagedView& pv, int S, int H, int sm_count) {
  if (S == 0) return 0;
  const AttnGeom gm = geometry(pv, H, sm_count);
  return ws_acc(gm.grid, gm.heads) + (int64_t)gm.grid * 2 * gm.heads * pv.D * 4;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a) {
  const AttnGeom gm = geometry(a.pv, a.H, a.sm_count);
  const bool two = head_tiles(a.pv, gm.G) == 2;
  if (a.pv.dtype == KVSEL_BF16) {
    if (a.pv.D == 128)
      return two ? launch<__nv_bfloat16, 128, 2>(a, gm) : launch<__nv_bfloat16, 128, 1>(a, gm);
    return two ? launch<__nv_bfloat16, 64, 2>(a, gm) : launch<__nv_bfloat16, 64, 1>(a, gm);
  }
  return a.pv.D == 128 ? launch<float, 128, 1>(a, gm) : launch<float, 64, 1>(a, gm);
}

}  // namespace kvsel
