// New tokens into a paged cache: per-head norm of queries and keys, position
// rotation, and the rows' places in the pages, in one pass.
//
// Mathematics, per token and head with the row x of D elements:
//   r_i = x_i * rsqrt(mean(x^2) + eps) * w_i                 (r = x without a weight)
//   (y_a, y_b) = scale * (r_a cos t - r_b sin t, r_b cos t + r_a sin t),  t = position * f_i
// for the pairs (a, b) = (i, i + rot/2), or (2i, 2i + 1) when interleaved; the rest of the
// row keeps r. fp32 throughout, one rounding at the store.
//
// Bound by memory: every row is read once and written once. What could get in the way is
// instructions, so a warp keeps one token's cosines and sines, times the norm's weights, for as
// many of its heads as leave the machine full, and a lane holds whole pairs: two 8-byte units of
// a head (D * size / 16 lanes a head), in the half layout one from either half, interleaved two
// neighbours. An element then costs a product and a sum, and no exchange between lanes but the
// norm's sum. (With 16 contiguous bytes a lane and the other half fetched by shuffles, 16384
// tokens took 105 us, 74% of the issue slots used.) The loads go through a ring of shared memory,
// seven heads' rows ahead without a register (four rows ahead in registers: 80 us): every lane
// copies what it will read itself, so nothing but its own copies is waited for.
#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 256;

// cos and sin of position * f, times scale. The angle in turns, position * f / (2 pi), is a
// sum of exact products: f / (2 pi) as two floats, the position as two parts of 16 bits, and
// every product with its own rounding error (fma). Whole turns drop out of each part without
// loss, so what is left is off by a few 2^-25 turns plus |position| 2^-47 turns; in fp32 alone
// the angle of position 10^6 would be off by 0.03.
__device__ __forceinline__ float fraction(float x) { return x - rintf(x); }

__device__ __forceinline__ void rotation(int position, float f, float scale, float* c, float* s) {
  const float inv_hi = 0.15915493667125702f;          // 1 / (2 pi) rounded to fp32
  const float inv_lo = 6.420638316725915e-9f;         // and the rest of it
  const float t_hi = f * inv_hi;
  const float t_lo = fmaf(f, inv_lo, fmaf(f, inv_hi, -t_hi));
  const float p_hi = (float)(position >> 16) * 65536.f, p_lo = (float)(position & 0xffff);
  const float a = p_hi * t_hi, ae = fmaf(p_hi, t_hi, -a);
  const float b = p_lo * t_hi, be = fmaf(p_lo, t_hi, -b);
  float turn = fraction(fraction(a) + fraction(b));
  turn += fraction(ae) + (be + fraction(fmaf(p_lo, t_lo, p_hi * t_lo)));
  sincospif(2.f * turn, s, c);
  *c *= scale;
  *s *= scale;
}

// An 8-byte unit: four bf16 or two fp32 values.
template <typename T>
__device__ __forceinline__ void unpack(const uint2& v, float* x) {
  if constexpr (sizeof(T) == 2) {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  } else {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
  }
}
template <typename T>
__device__ __forceinline__ uint2 pack(const float* x) {
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    return make_uint2(__float_as_uint(x[0]), __float_as_uint(x[1]));
  }
}

// Where token n's key and value rows go within a layer, in bytes; -1: nowhere.
__device__ __forceinline__ int64_t target_row(const AppendArgs& a, int n) {
  const int pos = a.cache_pos[n];
  if (pos < 0) return -1;
  const int col = pos >> a.pv.page_shift;
  int page = -1;
  if (!a.table) {
    if (col < a.pv.num_pages) page = col;
    else record_status(a.status, KVSEL_ERR_BAD_INDEX);
  } else {
    const int b = a.seqs ? a.seqs[n] : n;
    if (b >= 0 && b < a.num_seqs && col < a.table_width)
      page = checked_page(a.pv, a.table + (int64_t)b * a.table_width, col, a.status);
    else
      record_status(a.status, KVSEL_ERR_BAD_INDEX);
  }
  return page < 0 ? -1 : (int64_t)row_units(a.pv, page, pos & (a.pv.page_size - 1)) * kRowUnit;
}

__device__ __forceinline__ void copy8(uint32_t dst, const char* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// A warp takes `per_warp` passes of one (layer, token); a pass is 32 / kLanes heads of one
// kind: all of q's passes, then k's, then v's.
template <typename T, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const __grid_constant__ AppendArgs a,
                                                             int per_warp) {
  constexpr int U = 8 / sizeof(T), E = 2 * U;     // elements of a unit, of a lane
  constexpr int D = kLanes * E, kHeads = 32 / kLanes, kRowBytes = kLanes * 16;
  constexpr int kRing = 8;                        // passes in the ring
  __shared__ __align__(16) unsigned char ring[kRing][kThreads * 16];
  const int lane = threadIdx.x & 31, sub = lane % kLanes, grp = lane / kLanes;
  const int hk = a.src[1] ? a.pv.Hkv : 0;
  const int pq = (a.H + kHeads - 1) / kHeads, pk = (hk + kHeads - 1) / kHeads;
  const int passes = pq + 2 * pk, chunks = (passes + per_warp - 1) / per_warp;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= (int64_t)a.pv.layers * a.tokens * chunks) return;
  const int64_t lt = item / chunks;
  const int p0 = (int)(item - lt * chunks) * per_warp, p1 = min(passes, p0 + per_warp);
  const int layer = (int)(lt / a.tokens), n = (int)(lt - (int64_t)layer * a.tokens);

  // this lane's units of a head: (i, i + rot/2) for the lanes that turn in the half layout, two
  // neighbours else
  const int half = a.rot / 2, turning = a.rot / E;
  const bool turns = sub < turning;
  const bool apart = !kInterleaved && turns;
  const int ua = (apart ? sub : 2 * sub) * 8;     // byte offsets
  const int ub = apart ? ua + half * (int)sizeof(T) : ua + 8;

  const char* from[3];
#pragma unroll
  for (int i = 0; i < 3; ++i)
    from[i] = a.src[i] + layer * a.layer_bytes[i] + n * a.token_bytes[i] + grp * kRowBytes;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(&ring[0][threadIdx.x * 16]);
  auto issue = [&](int p) {
    if (p < p1) {
      const int kind = p < pq ? 0 : p < pq + pk ? 1 : 2;
      const int h0 = (p - (kind == 0 ? 0 : kind == 1 ? pq : pq + pk)) * kHeads;
      if (h0 + grp < (kind == 0 ? a.H : hk)) {
        const char* src = (kind == 0 ? from[0] : kind == 1 ? from[1] : from[2]) + h0 * kRowBytes;
        const uint32_t to = mine + ((p - p0) & (kRing - 1)) * (kThreads * 16);
        copy8(to, src + ua);
        copy8(to + 8, src + ub);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue(p0 + i);

  const int64_t row = p1 > pq ? target_row(a, n) : -1;
  float c[U], s[U];                               // of this lane's pairs
  const bool rotates = turns && p0 < pq + pk;
  if (rotates) {
    const int position = a.positions[n];
#pragma unroll
    for (int i = 0; i < U; ++i)
      rotation(position, a.inv_freq[sub * U + i], a.rope_scale, &c[i], &s[i]);
  }

  int p = p0;
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {
    const int first = kind == 0 ? 0 : kind == 1 ? pq : pq + pk;
    const int end = min(p1, kind == 0 ? pq : first + pk);
    if (p >= end) continue;
    const int heads = kind == 0 ? a.H : hk;
    char* dst = kind == 0 ? a.q_out + ((int64_t)layer * a.tokens + n) * a.H * kRowBytes
                          : (kind == 1 ? a.pv.k : a.pv.v) + layer * a.pv.layer_bytes + row;
    const bool placed = kind == 0 || row >= 0;
    const char* weight = kind == 0 ? a.weight[0] : kind == 1 ? a.weight[1] : nullptr;
    // the pair (x, y) becomes (x ca - y sb, y cb + x sa) g: cosines and sines times weights
    float ca[U], sa[U], cb[U], sb[U];
    if (kind < 2) {
      float w[E];
#pragma unroll
      for (int i = 0; i < E; ++i) w[i] = 1.f;
      if (weight) {
        const char* at = weight + (int64_t)layer * kRowBytes;
        unpack<T>(*reinterpret_cast<const uint2*>(at + ua), w);
        unpack<T>(*reinterpret_cast<const uint2*>(at + ub), w + U);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float wx = kInterleaved ? w[2 * i] : w[i], wy = kInterleaved ? w[2 * i + 1] : w[U + i];
        ca[i] = rotates ? wx * c[i] : wx;
        sa[i] = rotates ? wx * s[i] : 0.f;
        cb[i] = rotates ? wy * c[i] : wy;
        sb[i] = rotates ? wy * s[i] : 0.f;
      }
    }
#pragma unroll 2
    for (; p < end; ++p) {
      issue(p + kRing - 1);                       // into the slot that was read a pass ago
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      const uint4 v = shared16(mine + ((p - p0) & (kRing - 1)) * (kThreads * 16));
      const int h = (p - first) * kHeads + grp;
      uint2 ya = make_uint2(v.x, v.y), yb = make_uint2(v.z, v.w);
      if (kind < 2) {
        float x[E], r[E];
        unpack<T>(ya, x);
        unpack<T>(yb, x + U);
        float g = 1.f;
        if (weight) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
          for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          g = rsqrtf(ss * (1.f / D) + a.eps);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int ix = kInterleaved ? 2 * i : i, iy = kInterleaved ? 2 * i + 1 : U + i;
          r[ix] = x[ix] * ca[i];
          r[iy] = x[iy] * cb[i];
          if (turns) {                 // elsewhere an infinite neighbour must stay out
            r[ix] = fmaf(-x[iy], sb[i], r[ix]);
            r[iy] = fmaf(x[ix], sa[i], r[iy]);
          }
        }
        if (weight) {
#pragma unroll
          for (int i = 0; i < E; ++i) r[i] *= g;
        }
        ya = pack<T>(r);
        yb = pack<T>(r + U);
      }
      if (placed && h < heads) {
        char* to = dst + (int64_t)h * kRowBytes;
        *reinterpret_cast<uint2*>(to + ua) = ya;
        *reinterpret_cast<uint2*>(to + ub) = yb;
      }
    }
  }
}

template <typename T, int kLanes>
cudaError_t launch(const AppendArgs& a) {
  constexpr int kHeads = 32 / kLanes;
  const int hk = a.src[1] ? a.pv.Hkv : 0;
  const int passes = (a.H + kHeads - 1) / kHeads + 2 * ((hk + kHeads - 1) / kHeads);
  const int64_t rows = (int64_t)a.pv.layers * a.tokens;
  // passes a warp: one where there are few tokens (the longest chain counts), all of a token's
  // once that leaves 32 warps an SM
  int64_t per = rows * passes / ((int64_t)a.sm_count * 32);
  per = per < 1 ? 1 : per > passes ? passes : per;
  const int64_t warps = rows * ((passes + per - 1) / per);
  const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.interleaved)
    append_kernel<T, kLanes, true><<<(unsigned)blocks, kThreads, 0, a.stream>>>(a, (int)per);
  else
    append_kernel<T, kLanes, false><<<(unsigned)blocks, kThreads, 0, a.stream>>>(a, (int)per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a) {
  if (a.pv.dtype == KVSEL_BF16)
    return a.pv.D == 128 ? launch<__nv_bfloat16, 16>(a) : launch<__nv_bfloat16, 8>(a);
  return a.pv.D == 128 ? launch<float, 32>(a) : launch<float, 16>(a);
}

}  // namespace kvsel
