// One new query per (layer, sequence, query head) over a paged cache.
//
// Mathematics: s_j = q . k_j / sqrt(D) over the rows j < len, running maximum m and sum l of
// exp(s - m), out = sum_j exp(s_j - m) v_j / l, lse = m + ln l; an empty sequence has out = 0
// and lse = -inf. Base-2 units until the end.
//
// Bound by memory: every K and V row is read once for all the query heads that share it, so
// the products are small matrix products, S^T = K Q^T (16 rows x 8 heads a step) and
// O^T = V^T P^T, which fit mma.sync's m16n8 tile as they are: rows or dimensions are the 16,
// a group's heads the 8. (tcgen05 wants 128 rows and a trip through tensor memory for P; here
// the products take a small part of the time that a step's bytes take to arrive.) A dot product
// may take its dimensions in any order, so a lane's 32-byte pieces of K rows serve as the
// fragments, with q loaded in the same order; V's fragments pair two rows' values, which a byte
// permutation makes of two rows' pieces.
//
// Split: all (layer, sequence, head) instances' steps of 16 rows form one line, which the warps
// of one wave cut into equal parts, from the lengths on the device: a batch of any mix of lengths
// takes every SM the same time, and a single long sequence uses them all. A warp is on its own:
// it copies its rows into a ring of its own in shared memory (cp.async, two or more steps ahead,
// across the ends of instances too), needs no barrier, and writes an instance that it holds
// whole; of the others it writes a partial (max, sum, weighted values) to one of its two slots,
// and a second, dependent launch joins them in order (the same bits every time).
//
// Measured: 8 caches of 120000 to 131072 rows, 64 heads on 8, 4.09 GB: 600 to 615 us, 6.6 to
// 6.8 TB/s, the copy bandwidth; 48 caches of 0 to 8192 rows, 215 MB: 42 us, 75% of it; one cache
// of 293 rows: 8 us, two launches of dependent loads.
#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;                    // rows of a step
// What an instance's start and end cost, in steps: 48 sequences of 1 to 8192 rows took 77 us
// with 0, 49 with 1, 42.7 with 2, 42.5 with 3.
constexpr int kSegment = 2;
// Units that are worth a part of their own: one sequence of 293 rows took 9.7 us with 4, 8.1
// with 2.
constexpr int kLeast = 2;
constexpr int kJoinThreads = 128;  // small, so that a block for every warp of the first launch fits at once

// What the launch fixes; the rest follows from the lengths.
struct AttnGeom {
  int G;              // query heads per cache head
  int heads;          // query heads a warp takes
  int HG;             // head groups: ceil(G / heads)
  int grid;
};

// Workspace: the split instances that each warp has a piece of, the partials [warps][2][heads]:
// base-2 max and sum, and the weighted values [D]. An instance's first piece is in slot 1 of its
// warp, the others in slot 0.
struct SplitInfo {
  int64_t first_head; // index of its first query head in out / D, -1: none
  int first, last;    // the warps that have its pieces
  int heads, pad;
};
constexpr int kInfo = 2 * sizeof(SplitInfo);           // [0]: went on from an earlier warp, [1]: began here
__host__ __device__ inline int64_t ws_ml(int warps) { return kInfo * (int64_t)warps; }
__host__ __device__ inline int64_t ws_acc(int warps, int heads) {
  return ws_ml(warps) + ((16 * (int64_t)warps * heads + 15) & ~int64_t(15));
}

__device__ __forceinline__ void copy16(uint32_t dst, const char* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
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
// x = hi + lo in two tf32 values, 21 bits or more of x: hi rounded, so that what is cut off of lo
// has no common sign (it would shift every logit), in plain instructions where the conversions
// take several. NaN and infinities leave a NaN in lo.
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t* hi, uint32_t* lo) {
  *hi = (x + 0x1000u) & 0xffffe000u;
  *lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(*hi)) & 0xffffe000u;
}

// A warp's step: 16 rows x 8 * NT heads. Lane (g, t) = (lane / 4, lane % 4) holds of S^T rows g
// and g + 8, heads 2t and 2t + 1; of O^T (m-tile i) dimensions g * D/8 + 2i and + 1, heads 2t and
// 2t + 1. It reads of K rows g, g + 8 the 32-byte pieces t, t + 4, .., of V rows 2t, 2t + 1,
// 2t + 8, 2t + 9 the D/8 dimensions from g * D/8 on.
template <typename T, int D, int NT>
struct Step {
  static constexpr int kEb = sizeof(T);
  static constexpr int kRowBytes = D * kEb;
  static constexpr int kHalf = kRows * kRowBytes;     // a step's K, or V
  static constexpr int kStage = 2 * kHalf;
  // steps in the ring: with the warps an SM holds, some 160 KB
  static constexpr int kStages = kStage == 4096 ? 5 : 3;
  static constexpr int kBlocks = kStage == 16384 ? 1 : 2;    // blocks an SM
  static constexpr int kKw = kRowBytes / 16;          // words of a K row a lane reads
  static constexpr int kVq = kRowBytes / 128;         // 16-byte units of a V row a lane reads
  static constexpr int kMt = D / 16;                  // m-tiles of O^T
  static constexpr int kQ = kKw * (kEb == 2 ? 1 : 2); // words of q's fragments, per 8 heads
  uint32_t qf[NT][kQ];
  float o[NT][kMt][4];
  float m[NT][2], l[NT][2];

  // 16-byte unit u of row r lies at unit u ^ swizzle(r) of its row: the eight lanes of a
  // shared-memory access (two rows' pieces of K; four rows' of V) then touch all banks once.
  static __device__ __forceinline__ int swizzle_k(int r) { return r & 1; }
  static __device__ __forceinline__ int swizzle_v(int r) {
    const int t = (r >> 1) & 3;
    return kVq == 1 ? 2 * t : kVq == 2 ? (t & 1) | (t & 2) << 1 : t;
  }

  __device__ __forceinline__ void issue(uint32_t stage, const char* kb, const char* vb, uint32_t off,
                                        int lane) const {
    constexpr int kLanes = kRowBytes / 16;            // lanes a row
    const int unit = lane % kLanes;
#pragma unroll
    for (int r0 = 0; r0 < kRows; r0 += 32 / kLanes) {
      const int r = r0 + lane / kLanes;
      const int64_t at = (int64_t)__shfl_sync(0xffffffffu, off, r) * kRowUnit + unit * 16;
      const uint32_t row = stage + r * kRowBytes;
      copy16(row + ((unit ^ swizzle_k(r)) << 4), kb + at);
      copy16(row + kHalf + ((unit ^ swizzle_v(r)) << 4), vb + at);
    }
  }

  // q in the order of K's pieces; heads past the group's are zero
  struct Query {
    uint4 w[NT][kKw / 4];
  };
  static __device__ __forceinline__ void fetch(Query& f, const char* q, int n_heads, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int c = 0; c < kKw / 4; ++c) {             // 16 bytes at a time
        f.w[x][c] = make_uint4(0, 0, 0, 0);
        if (x * 8 + g < n_heads)
          f.w[x][c] = *reinterpret_cast<const uint4*>(q + (int64_t)(x * 8 + g) * kRowBytes +
                                                      (c >> 1) * 128 + t * 32 + (c & 1) * 16);
      }
  }
  __device__ __forceinline__ void begin(const Query& f) {
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int c = 0; c < kKw / 4; ++c) {
        const uint4 w = f.w[x][c];
        if constexpr (kEb == 2) {
          qf[x][4 * c] = w.x;
          qf[x][4 * c + 1] = w.y;
          qf[x][4 * c + 2] = w.z;
          qf[x][4 * c + 3] = w.w;
        } else {                                      // hi, hi, lo, lo of every two
          split_tf32(w.x, &qf[x][8 * c], &qf[x][8 * c + 2]);
          split_tf32(w.y, &qf[x][8 * c + 1], &qf[x][8 * c + 3]);
          split_tf32(w.z, &qf[x][8 * c + 4], &qf[x][8 * c + 6]);
          split_tf32(w.w, &qf[x][8 * c + 5], &qf[x][8 * c + 7]);
        }
      }
#pragma unroll
      for (int i = 0; i < kMt; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[x][i][k] = 0.f;
      m[x][0] = m[x][1] = -INFINITY;
      l[x][0] = l[x][1] = 0.f;
    }
  }

  // S^T of this step's rows and heads.
  __device__ __forceinline__ void scores(float (&s)[NT][4], uint32_t stage, int lane) const {
    const int g = lane >> 2, t = lane & 3;
    constexpr int kAcc = 4;                      // short chains: the matrix unit cuts off at every link
    float acc[NT][kAcc][4] = {};
    const uint32_t row = stage + g * kRowBytes;
#pragma unroll
    for (int c = 0; c < kKw / 4; ++c) {
      const uint32_t at = row + ((((c >> 1) * 8 + 2 * t + (c & 1)) ^ swizzle_k(g)) << 4);
      const uint4 a = shared16(at), b = shared16(at + 8 * kRowBytes);
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        if constexpr (kEb == 2) {
          mma_bf16(acc[x][(2 * c) % kAcc], a.x, b.x, a.y, b.y, qf[x][4 * c], qf[x][4 * c + 1]);
          mma_bf16(acc[x][(2 * c + 1) % kAcc], a.z, b.z, a.w, b.w, qf[x][4 * c + 2], qf[x][4 * c + 3]);
        } else {
          const uint32_t e[2][4] = {{a.x, b.x, a.y, b.y}, {a.z, b.z, a.w, b.w}};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t h[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split_tf32(e[k][i], &h[i], &w[i]);
            const uint32_t* f = &qf[x][8 * c + 4 * k];
            mma_tf32(acc[x][k], h[0], h[1], h[2], h[3], f[0], f[1]);
            mma_tf32(acc[x][2], w[0], w[1], w[2], w[3], f[0], f[1]);
            mma_tf32(acc[x][3], h[0], h[1], h[2], h[3], f[2], f[3]);
          }
        }
      }
    }
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int w = kAcc / 2; w > 0; w /= 2)
#pragma unroll
          for (int k = 0; k < w; ++k) acc[x][k][i] += acc[x][k + w][i];
        s[x][i] = acc[x][0][i];
      }
  }

  // Running maximum and sum; s becomes the weights, f the factors of what was there before.
  __device__ __forceinline__ void weigh(float (&s)[NT][4], float (&f)[NT][2], uint32_t valid,
                                        float scale, int lane) {
    const int g = lane >> 2;
    const bool ok0 = valid >> g & 1u, ok1 = valid >> (g + 8) & 1u;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        s[x][c] = ok0 ? s[x][c] * scale : -INFINITY;
        s[x][2 + c] = ok1 ? s[x][2 + c] * scale : -INFINITY;
        float mx = fmaxf(s[x][c], s[x][2 + c]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        mx = fmaxf(mx, m[x][c]);
        const float ref = mx == -INFINITY ? 0.f : mx;
        f[x][c] = ex2(m[x][c] - ref);
        m[x][c] = mx;
        // -inf gives 0; NaN (and +inf, whose maximum it is) gives NaN
        s[x][c] = ex2(s[x][c] - ref);
        s[x][2 + c] = ex2(s[x][2 + c] - ref);
        l[x][c] = fmaf(l[x][c], f[x][c], s[x][c] + s[x][2 + c]);
      }
  }

  // O^T = O^T f + V^T P^T; p: this lane's weights, in S^T's places. The product of a step is
  // formed from zero and added in fp32: the matrix unit cuts off what it adds to, and over the
  // thousands of steps of a long cache that cost 2e-5 of the result.
  __device__ __forceinline__ void add(float (&to)[4], const float (&f)[2], const float (&d)[4]) {
    const Two ff = two(f[0], f[1]);
    const float2 a = both(fma(two(to[0], to[1]), ff, two(d[0], d[1])));
    const float2 b = both(fma(two(to[2], to[3]), ff, two(d[2], d[3])));
    to[0] = a.x;
    to[1] = a.y;
    to[2] = b.x;
    to[3] = b.y;
  }
  __device__ __forceinline__ void values(const float (&p)[NT][4], const float (&f)[NT][2], uint32_t stage,
                                         int lane) {
    const int g = lane >> 2, t = lane & 3;
    uint32_t bh[NT][kEb], bl[NT][kEb], br[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float p0 = p[x][2 * i], p1 = p[x][2 * i + 1];
        if constexpr (kEb == 2) {
          // weights as a sum of three bf16, 24 bits: with two the results were off by 1e-6, with
          // one by 1e-3, and the time is the same
          const uint32_t hi = pack_bf16(p0, p1);
          const float p2 = p0 - __uint_as_float(hi << 16), p3 = p1 - __uint_as_float(hi & 0xffff0000u);
          const uint32_t lo = pack_bf16(p2, p3);
          const uint32_t rest = pack_bf16(p2 - __uint_as_float(lo << 16),
                                          p3 - __uint_as_float(lo & 0xffff0000u));
          bh[x][i] = transposed(hi);
          bl[x][i] = transposed(lo);
          br[x][i] = transposed(rest);
        } else {
          // transposed in two halves; then rows 2t, 2t + 1 (+ 8) of head g
          const uint32_t u = __float_as_uint(p0), w = __float_as_uint(p1);
          const uint32_t top = transposed(__byte_perm(u, w, 0x7632));
          const uint32_t low = transposed(__byte_perm(u, w, 0x5410));
          split_tf32(__byte_perm(low, top, 0x5410), &bh[x][2 * i], &bl[x][2 * i]);
          split_tf32(__byte_perm(low, top, 0x7632), &bh[x][2 * i + 1], &bl[x][2 * i + 1]);
        }
      }
    const uint32_t row = stage + kHalf + 2 * t * kRowBytes;
#pragma unroll
    for (int c = 0; c < kVq; ++c) {
      const uint32_t at = row + (((g * kVq + c) ^ swizzle_v(2 * t)) << 4);   // 2t + 1, + 8, + 9 alike
      const uint4 r0 = shared16(at), r1 = shared16(at + kRowBytes), r2 = shared16(at + 8 * kRowBytes),
                  r3 = shared16(at + 9 * kRowBytes);
      const uint32_t v[4][4] = {{r0.x, r0.y, r0.z, r0.w}, {r1.x, r1.y, r1.z, r1.w},
                                {r2.x, r2.y, r2.z, r2.w}, {r3.x, r3.y, r3.z, r3.w}};
      if constexpr (kEb == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = __byte_perm(v[0][i], v[1][i], 0x5410);
          const uint32_t a1 = __byte_perm(v[0][i], v[1][i], 0x7632);
          const uint32_t a2 = __byte_perm(v[2][i], v[3][i], 0x5410);
          const uint32_t a3 = __byte_perm(v[2][i], v[3][i], 0x7632);
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            float d[4] = {};
            mma_bf16(d, a0, a1, a2, a3, br[x][0], br[x][1]);
            mma_bf16(d, a0, a1, a2, a3, bl[x][0], bl[x][1]);
            mma_bf16(d, a0, a1, a2, a3, bh[x][0], bh[x][1]);
            add(o[x][c * 4 + i], f[x], d);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float d[NT][4] = {};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t h[4], w[4];
            split_tf32(v[2 * k][2 * i], &h[0], &w[0]);
            split_tf32(v[2 * k][2 * i + 1], &h[1], &w[1]);
            split_tf32(v[2 * k + 1][2 * i], &h[2], &w[2]);
            split_tf32(v[2 * k + 1][2 * i + 1], &h[3], &w[3]);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              mma_tf32(d[x], h[0], h[1], h[2], h[3], bh[x][2 * k], bh[x][2 * k + 1]);
              mma_tf32(d[x], w[0], w[1], w[2], w[3], bh[x][2 * k], bh[x][2 * k + 1]);
              mma_tf32(d[x], h[0], h[1], h[2], h[3], bl[x][2 * k], bl[x][2 * k + 1]);
            }
          }
#pragma unroll
          for (int x = 0; x < NT; ++x) add(o[x][c * 2 + i], f[x], d[x]);
        }
      }
    }
  }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, Step<T, D, NT>::kBlocks)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ AttnGeom gm) {
  using St = Step<T, D, NT>;
  extern __shared__ __align__(128) unsigned char smem[];   // rings, valid rows of their steps, pre
  __shared__ int warp_sums[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint32_t* const valid = reinterpret_cast<uint32_t*>(smem + kWarps * St::kStages * St::kStage) +
                          warp * St::kStages;
  int* const pre = reinterpret_cast<int*>(smem + kWarps * St::kStages * (St::kStage + 4));
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (St::kStages * St::kStage);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // units before every sequence: its steps, and kSegment more that stand for an instance's start
  // and end (a part of many short instances would take far longer than one of a long one)
  const int max_rows = a.table_width << a.pv.page_shift;
  int nb = 0;
  for (int b0 = 0; b0 < a.S; b0 += kThreads) {
    const int b = b0 + tid;
    int x = 0;
    if (b < a.S) {
      const int len = checked_len(a.lens[b], max_rows, a.status);
      x = len ? (int)(((int64_t)len + kRows - 1) / kRows) + kSegment : 0;
    }
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

  // this warp's part of the line
  const int HH = a.pv.Hkv * gm.HG, warps = gm.grid * kWarps;
  const int64_t per_layer = (int64_t)nb * HH;
  const int64_t units = per_layer * a.pv.layers;
  const int parts = (int)min((int64_t)warps, (units + kLeast - 1) / kLeast);
  const int part = blockIdx.x * kWarps + warp;
  // the first `longer` parts have a unit more than the others
  const int64_t each = parts ? quotient(units, parts) : 0;
  const int longer = (int)(units - each * parts);
  auto part_start = [&](int64_t c) { return c * each + min(c, (int64_t)longer); };
  auto part_of = [&](int64_t unit) {
    const int64_t split = (each + 1) * longer;
    return (int)(unit < split ? quotient(unit, each + 1) : longer + quotient(unit - split, each));
  };
  const bool works = part < parts;
  const int64_t u0 = works ? part_start(part) : 0, u1 = works ? part_start(part + 1) : 0;

  // The instance at unit u of this part, and its steps [first, last) within the part: none where
  // the part ends before the instance's first step.
  struct Place {
    int layer, b, head, first, last, n_steps;
    int64_t end;              // of the instance, or of the part
  };
  auto locate = [&](int64_t u) {
    Place x;
    x.layer = a.pv.layers == 1 ? 0 : (int)quotient(u, per_layer);
    const int64_t rem = u - x.layer * per_layer;
    x.b = upper_find(a.S, (int)quotient(rem, HH), [&](int i) { return pre[i]; });
    const int n = pre[x.b + 1] - pre[x.b];
    const int64_t local = rem - (int64_t)pre[x.b] * HH;
    x.head = (int)quotient(local, n);
    const int at = (int)(local - (int64_t)x.head * n);
    x.end = min(u + (n - at), u1);
    x.n_steps = n - kSegment;
    x.first = max(0, at - kSegment);
    x.last = max(0, at + (int)(x.end - u) - kSegment);
    return x;
  };

  // the copying side: the instance that it is in, and this lane's row and table entry for the
  // next step to copy
  int64_t pu = u0;                        // unit after that instance
  int p_left = 0, p_row = 0, p_len = 0, p_page = -1;
  const int32_t* p_table = nullptr;
  int64_t p_base = 0;
  auto look = [&] {
    while (p_left == 0 && pu < u1) {
      const Place x = locate(pu);
      pu = x.end;
      p_left = x.last - x.first;
      p_row = x.first * kRows + (lane & 15);
      p_len = min(max(a.lens[x.b], 0), max_rows);
      p_table = a.table + (int64_t)x.b * a.table_width;
      p_base = x.layer * a.pv.layer_bytes + (int64_t)quotient(x.head, gm.HG) * a.pv.head_units * kRowUnit;
    }
    if (p_left) p_page = p_row < p_len ? __ldg(p_table + (p_row >> a.pv.page_shift)) : -1;
  };
  St st;
  auto copy_step = [&](int slot) {
    if (p_left) {
      const bool in = p_row < p_len;
      const bool ok = in && p_page >= 0 && p_page < a.pv.num_pages;
      if (in && !ok) record_status(a.status, KVSEL_ERR_BAD_INDEX);
      const uint32_t v = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      uint32_t off = ok ? row_units(a.pv, p_page, p_row & (a.pv.page_size - 1)) : 0;
      // rows that do not count are copies of one that does: nothing else may be read
      const uint32_t other = __shfl_sync(0xffffffffu, off, v ? __ffs(v) - 1 : 0);
      off = ok ? off : other;
      if (v) st.issue(ring + slot * St::kStage, a.pv.k + p_base, a.pv.v + p_base, off, lane);
      if (lane == 0) valid[slot] = v;
      p_row += kRows;
      --p_left;
      look();
    }
    copies_commit();
  };

  // lane 0's own, so that a later one comes after
  SplitInfo* const info = reinterpret_cast<SplitInfo*>(a.ws) + 2 * part;
  if (lane == 0) info[0].first_head = info[1].first_head = -1;
  float2* const ml = reinterpret_cast<float2*>(a.ws + ws_ml(warps));
  float* const acc = reinterpret_cast<float*>(a.ws + ws_acc(warps, gm.heads));

  look();
#pragma unroll
  for (int i = 0; i < St::kStages - 1; ++i) copy_step(i);
  int slot = 0;
  // the next instance with steps in this part, and its heads' queries
  Place x{};
  typename St::Query query;
  int64_t u = u0, first_head = 0;
  int n_heads = 0;
  auto next = [&] {
    x.first = x.last = 0;
    while (x.first == x.last && u < u1) {
      x = locate(u);
      if (x.first == x.last) u = x.end;
    }
    if (x.first == x.last) return;
    const int kvh = (int)quotient(x.head, gm.HG), hg = x.head - kvh * gm.HG;
    n_heads = min(gm.heads, gm.G - hg * gm.heads);
    first_head = ((int64_t)x.layer * a.S + x.b) * a.H + kvh * gm.G + hg * gm.heads;
    St::fetch(query, static_cast<const char*>(a.q) + first_head * St::kRowBytes, n_heads, lane);
  };
  next();
  while (x.first < x.last) {
    st.begin(query);
    for (int i = x.first; i < x.last; ++i) {
      copies_wait<St::kStages - 2>();
      __syncwarp();                    // every lane's copies are there, and the step before is read
      copy_step(slot == 0 ? St::kStages - 1 : slot - 1);
      const uint32_t stage = ring + slot * St::kStage, v = valid[slot];
      if (v) {
        float s[NT][4], f[NT][2];
        st.scores(s, stage, lane);
        st.weigh(s, f, v, a.scale_log2, lane);
        st.values(s, f, stage, lane);
      }
      slot = slot == St::kStages - 1 ? 0 : slot + 1;
    }

    const bool begins = x.first == 0, whole = begins && x.last == x.n_steps;
    const int64_t at = ((int64_t)part * 2 + (begins ? 1 : 0)) * gm.heads;
    const int64_t first = first_head;
    const int heads = n_heads;
    if (!whole && lane == 0) {
      // a piece that goes on starts with step x.first; the instance ends after its last step
      const int64_t stop = x.end + (x.n_steps - x.last);
      info[begins ? 1 : 0] = SplitInfo{first, begins ? part : part_of(u - x.first), part_of(stop - 1),
                                       heads, 0};
    }
    u = x.end;
    next();                            // its queries arrive while this one's results go out
    bool bad = false;
#pragma unroll
    for (int y = 0; y < NT; ++y)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = st.l[y][c];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int h = y * 8 + 2 * t + c;
        if (h >= heads) continue;
        const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
        float4* to = reinterpret_cast<float4*>((whole ? a.out + (first + h) * D : acc + (at + h) * D) +
                                               g * (D / 8));
        if (whole) bad |= !finite_f(l);
#pragma unroll
        for (int i = 0; i < St::kMt; i += 2) {
          const float4 w = make_float4(st.o[y][i][c] * inv, st.o[y][i][2 + c] * inv,
                                       st.o[y][i + 1][c] * inv, st.o[y][i + 1][2 + c] * inv);
          if (whole) bad |= !finite_f(w.x) || !finite_f(w.y) || !finite_f(w.z) || !finite_f(w.w);
          to[i / 2] = w;
        }
        if (g == 0 && !whole) ml[at + h] = make_float2(st.m[y][c], l);
        if (g == 0 && whole && a.lse)
          a.lse[first + h] = l == 0.f ? -INFINITY : (st.m[y][c] + log2f(l)) * 0.6931471805599453f;
      }
    if (bad) record_status(a.status, KVSEL_ERR_NONFINITE);
  }
}

// Joins the split instances' pieces. An instance that spans the parts first .. last is joined by
// the blocks first .. last, which share out its heads, or quarters of its heads' values. A block's warps share its items (of the instance that goes on in
// its part and of the one that begins there), and the pieces of an item where there are fewer
// items than warps; within a warp, as many lanes as the item's values need take a piece. Every
// lane group keeps a maximum of its own, so that one pass over the pieces does.
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 8) paged_join_kernel(const __grid_constant__ PagedAttnArgs a,
                                                                     const __grid_constant__ AttnGeom gm) {
  constexpr int kJoinWarps = kJoinThreads / 32, kAhead = 4;
  __shared__ float maxs[kJoinWarps], sums[kJoinWarps];
  __shared__ float4 vals[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = gm.grid * kWarps;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float2* ml = reinterpret_cast<const float2*>(a.ws + ws_ml(warps));
  const float* acc = reinterpret_cast<const float*>(a.ws + ws_acc(warps, gm.heads));
  const SplitInfo* infos = reinterpret_cast<const SplitInfo*>(a.ws) + 2 * blockIdx.x;
  const SplitInfo on = infos[0], begun = infos[1];
  // log2 of the parts that a head's values are joined in: four where the pieces are many (24
  // heads of 1216 pieces: 41 us for the call, 71 without), one where they are few (0.5 us less);
  // and the items that are this block's: its place among the instance's blocks, then every n-th
  auto slices = [](const SplitInfo& i) {
    const int n = i.last - i.first + 1;
    return n >= 64 && n >= 4 * i.heads ? 2 : 0;
  };
  auto share = [&](const SplitInfo& i) {
    if (i.first_head < 0) return 0;           // nothing else of it is written
    const int n = i.last - i.first + 1, at = (int)blockIdx.x - i.first;
    const int items = i.heads << slices(i);
    return at >= items ? 0 : (items - at + n - 1) / n;
  };
  const int count0 = share(on), count = count0 + share(begun);
  if (count == 0) return;
  int per = kJoinWarps;                       // warps an item: a power of two
  while (per > 1 && per * count > kJoinWarps) per >>= 1;
  const int sub = warp & (per - 1);
  for (int c0 = 0; c0 < count; c0 += kJoinWarps / per) {
    const int c = c0 + warp / per;
    const SplitInfo& info = c < count0 ? on : begun;
    const int n = info.last - info.first + 1, shift = slices(info);
    const int item = (int)blockIdx.x - info.first + (c < count0 ? c : c - count0) * n;
    const int lane_shift = (D == 128 ? 5 : 4) - shift;         // lanes a piece: 4 values each
    const int h = item >> shift, lanes = 1 << lane_shift;
    const int place = lane & (lanes - 1), groups = 32 >> lane_shift, grp = lane >> lane_shift;
    const int d = ((item & ((1 << shift) - 1)) * lanes + place) * 4;
    float mx = -INFINITY, sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < count) {
      const int step = per * groups;
      for (int i0 = sub * groups + grp; i0 < n; i0 += step * kAhead) {
        float2 y[kAhead];
        float4 w[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + k * step;
          const int64_t at = ((int64_t)(info.first + i) * 2 + (i == 0 ? 1 : 0)) * gm.heads + h;
          y[k] = make_float2(-INFINITY, 0.f);
          w[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < n) {
            y[k] = ml[at];
            w[k] = *reinterpret_cast<const float4*>(acc + at * D + d);
          }
        }
        float top = mx;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) top = fmaxf(top, y[k].x);
        const float ref = top == -INFINITY ? 0.f : top, f = ex2(mx - ref);
        mx = top;
        sum *= f;
        v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float p = ex2(y[k].x - ref);        // of -inf: 0; a NaN sum stays NaN
          sum = fmaf(y[k].y, p, sum);
          v = make_float4(fmaf(w[k].x, p, v.x), fmaf(w[k].y, p, v.y), fmaf(w[k].z, p, v.z),
                          fmaf(w[k].w, p, v.w));
        }
      }
    }
    // the lane groups' results, added in pairs
    for (int off = lanes; off < 32; off <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, mx, off), so = __shfl_xor_sync(0xffffffffu, sum, off);
      const float4 vo = make_float4(__shfl_xor_sync(0xffffffffu, v.x, off), __shfl_xor_sync(0xffffffffu, v.y, off),
                                    __shfl_xor_sync(0xffffffffu, v.z, off), __shfl_xor_sync(0xffffffffu, v.w, off));
      const float top = fmaxf(mx, mo), ref = top == -INFINITY ? 0.f : top;
      const float f = ex2(mx - ref), fo = ex2(mo - ref);
      mx = top;
      sum = sum * f + so * fo;
      v = make_float4(v.x * f + vo.x * fo, v.y * f + vo.y * fo, v.z * f + vo.z * fo, v.w * f + vo.w * fo);
    }
    __syncthreads();                          // the items before have been read
    if (lane == 0) {
      maxs[warp] = mx;
      sums[warp] = sum;
    }
    if (grp == 0) vals[warp][place] = v;
    __syncthreads();
    if (sub != 0 || c >= count || grp != 0) continue;
    float top = mx;
    for (int w = 1; w < per; ++w) top = fmaxf(top, maxs[warp + w]);
    const float ref = top == -INFINITY ? 0.f : top;
    float total = 0.f;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < per; ++w) {
      const float f = ex2(maxs[warp + w] - ref);
      const float4 x = vals[warp + w][place];
      total = fmaf(sums[warp + w], f, total);
      r = make_float4(fmaf(x.x, f, r.x), fmaf(x.y, f, r.y), fmaf(x.z, f, r.z), fmaf(x.w, f, r.w));
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    r = make_float4(r.x * inv, r.y * inv, r.z * inv, r.w * inv);
    *reinterpret_cast<float4*>(a.out + (info.first_head + h) * D + d) = r;
    if (d == 0 && a.lse)
      a.lse[info.first_head + h] = total == 0.f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
    if (!finite_f(total) || !finite_f(r.x) || !finite_f(r.y) || !finite_f(r.z) || !finite_f(r.w))
      record_status(a.status, KVSEL_ERR_NONFINITE);
  }
}

// Tiles of 8 heads a warp: in bf16 up to three (a row's fragments then serve three products), as
// many as read the rows the fewest times (24 heads a group: 149 us with three, where two tiles
// read the rows twice in 200); fp32's split fragments leave registers for one.
int head_tiles(const PagedView& pv, int G) {
  if (pv.dtype == KVSEL_F32) return 1;
  int best = 1;
  auto reads = [&](int nt) { return (G + 8 * nt - 1) / (8 * nt); };
  for (int nt = 2; nt <= 3; ++nt)
    if (reads(nt) < reads(best)) best = nt;
  return best;
}

template <typename T, int D, int NT>
int smem_bytes(int S) {
  using St = Step<T, D, NT>;
  return kWarps * St::kStages * (St::kStage + 4) + (S + 1) * (int)sizeof(int);
}

AttnGeom geometry(const PagedView& pv, int H, int sm_count) {
  AttnGeom gm;
  gm.G = H / pv.Hkv;
  const int most = 8 * head_tiles(pv, gm.G);
  gm.HG = (gm.G + most - 1) / most;
  gm.heads = (gm.G + gm.HG - 1) / gm.HG;
  gm.grid = sm_count * (pv.dtype == KVSEL_F32 && pv.D == 128 ? Step<float, 128, 1>::kBlocks
                                                             : Step<__nv_bfloat16, 128, 1>::kBlocks);
  return gm;
}

template <typename T, int D, int NT>
cudaError_t launch(const PagedAttnArgs& a, const AttnGeom& gm) {
  static_assert(kWarps * Step<T, D, NT>::kStages * (Step<T, D, NT>::kStage + 4) +
                        (kMaxPagedSeqs + 1) * 4 + 64 <= 227 * 1024, "ring and steps fit shared memory");
  // always the same value: another thread's call may come between
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<T, D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem_bytes<T, D, NT>(kMaxPagedSeqs));
  if (e) return e;
  paged_attn_kernel<T, D, NT><<<gm.grid, kThreads, smem_bytes<T, D, NT>(a.S), a.stream>>>(a, gm);
  if ((e = cudaGetLastError())) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(gm.grid * kWarps));
  cfg.blockDim = dim3(kJoinThreads);
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
  const int warps = gm.grid * kWarps;
  return ws_acc(warps, gm.heads) + (int64_t)warps * 2 * gm.heads * pv.D * 4;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a) {
  const AttnGeom gm = geometry(a.pv, a.H, a.sm_count);
  const int nt = head_tiles(a.pv, gm.G);
  if (a.pv.dtype == KVSEL_BF16) {
    if (a.pv.D == 128)
      return nt == 3   ? launch<__nv_bfloat16, 128, 3>(a, gm)
             : nt == 2 ? launch<__nv_bfloat16, 128, 2>(a, gm)
                       : launch<__nv_bfloat16, 128, 1>(a, gm);
    return nt == 3   ? launch<__nv_bfloat16, 64, 3>(a, gm)
           : nt == 2 ? launch<__nv_bfloat16, 64, 2>(a, gm)
                     : launch<__nv_bfloat16, 64, 1>(a, gm);
  }
  return a.pv.D == 128 ? launch<float, 128, 1>(a, gm) : launch<float, 64, 1>(a, gm);
}

}  // namespace kvsel
