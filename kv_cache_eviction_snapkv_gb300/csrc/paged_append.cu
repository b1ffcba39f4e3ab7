// New tokens into a paged cache: per-head norm of queries and keys, position
// rotation, and the rows' places in the pages, in one pass.
//
// Mathematics, per token and head with the row x of D elements:
//   r_i = x_i * rsqrt(mean(x^2) + eps) * w_i                 (r = x without a weight)
//   (y_a, y_b) = scale * (r_a cos t - r_b sin t, r_b cos t + r_a sin t),  t = position * f_i
// for the pairs (a, b) = (i, i + rot/2), or (2i, 2i + 1) when interleaved; the rest of the
// row keeps r. fp32 throughout, one rounding at the store.
//
// Bound by memory: every row is read once and written once. What could get in the way is the
// sines, so a warp keeps one token's for as many of its heads as leave the machine full: a lane
// holds 16 bytes of a head (D * size / 16 lanes a head) and so needs the same few pairs for every
// head; per head it is then two products and a sum an element, with the weight multiplied into
// the cosine and sine. A pair's other element comes from another lane (half layout; rot / 2 is a
// whole number of lanes) or the same one (interleaved).
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

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[16 / sizeof(T)]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[16 / sizeof(T)]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      w[i] = __float_as_uint(x[i]);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
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

// A warp takes `per_warp` passes of one (layer, token); a pass is 32 / kLanes heads of one
// kind: all of q's passes, then k's, then v's.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const __grid_constant__ AppendArgs a,
                                                             int per_warp) {
  constexpr int E = 16 / sizeof(T);               // elements a lane holds of a head
  constexpr int D = kLanes * E, kHeads = 32 / kLanes, kRowBytes = kLanes * 16;
  constexpr int kAhead = 4;                       // passes whose loads go out together
  __shared__ float turn[2 * E][kThreads];         // every lane's own cosines and sines
  const int lane = threadIdx.x & 31, sub = lane % kLanes, grp = lane / kLanes;
  const int hk = a.src[1] ? a.pv.Hkv : 0;
  const int pq = (a.H + kHeads - 1) / kHeads, pk = (hk + kHeads - 1) / kHeads;
  const int passes = pq + 2 * pk, chunks = (passes + per_warp - 1) / per_warp;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= (int64_t)a.pv.layers * a.tokens * chunks) return;
  const int64_t lt = item / chunks;
  const int p0 = (int)(item - lt * chunks) * per_warp, p1 = min(passes, p0 + per_warp);
  const int layer = (int)(lt / a.tokens), n = (int)(lt - (int64_t)layer * a.tokens);

  auto head_of = [&](int p, int* kind) {
    *kind = p < pq ? 0 : p < pq + pk ? 1 : 2;
    return (p - (*kind == 0 ? 0 : *kind == 1 ? pq : pq + pk)) * kHeads + grp;
  };
  auto source = [&](int kind, int h) {
    return reinterpret_cast<const uint4*>(a.src[kind] + layer * a.layer_bytes[kind] +
                                          n * a.token_bytes[kind] + h * kRowBytes + sub * 16);
  };
  auto load = [&](uint4 (&v)[kAhead], int p) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      int kind;
      const int h = head_of(p + u, &kind);
      v[u] = make_uint4(0, 0, 0, 0);
      if (p + u < p1 && h < (kind == 0 ? a.H : hk)) v[u] = __ldcs(source(kind, h));
    }
  };
  uint4 v[kAhead];
  load(v, p0);

  const int64_t row = p1 > pq ? target_row(a, n) : -1;
  // this lane's cosines and sines; sin with the sign of its own element
  const int half = a.rot / 2, e0 = sub * E;
  const bool turns = e0 < a.rot;
  const bool cross = turns && !a.interleaved;     // the other elements are in another lane
  const int other_lane = cross ? lane + (e0 < half ? half : -half) / E : lane;
  float wa[E], wb[E];
  if (turns && p0 < pq + pk) {
    const int position = a.positions[n];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = e0 + i;
      const int pair = a.interleaved ? e >> 1 : e < half ? e : e - half;
      float c, s;
      rotation(position, a.inv_freq[pair], a.rope_scale, &c, &s);
      turn[i][threadIdx.x] = c;
      turn[E + i][threadIdx.x] = (a.interleaved ? i % 2 == 0 : e < half) ? -s : s;
    }
  }

  int have = -1;                                  // kind that wa, wb are for
  for (int p = p0; p < p1; p += kAhead) {
    if (p > p0) load(v, p);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (p + u >= p1) break;
      int kind;
      const int h = head_of(p + u, &kind);
      const bool live = h < (kind == 0 ? a.H : hk);
      char* dst = kind == 0 ? a.q_out + (((int64_t)layer * a.tokens + n) * a.H + h) * kRowBytes
                            : (kind == 1 ? a.pv.k : a.pv.v) + layer * a.pv.layer_bytes + row +
                                  (int64_t)h * kRowBytes;
      uint4 y = v[u];
      if (kind < 2) {
        const char* weight = kind == 0 ? a.weight[0] : a.weight[1];
        if (kind != have) {
          // y = g (x wa + other wb): weight times cosine, the other's weight times sine
          have = kind;
          float w[E];
#pragma unroll
          for (int i = 0; i < E; ++i) w[i] = 1.f;
          if (weight)
            unpack<T>(*reinterpret_cast<const uint4*>(weight + (int64_t)layer * kRowBytes + sub * 16), w);
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const float away = __shfl_sync(0xffffffffu, w[i], other_lane);
            wa[i] = turns ? w[i] * turn[i][threadIdx.x] : w[i];
            wb[i] = turns ? (cross ? away : w[i ^ 1]) * turn[E + i][threadIdx.x] : 0.f;
          }
        }
        float x[E], o[E];
        unpack<T>(v[u], x);
        float g = 1.f;
        if (weight) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
          for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          g = rsqrtf(ss * (1.f / D) + a.eps);
        }
        if (a.rot > 0 && !a.interleaved) {
          const uint4 far = make_uint4(__shfl_sync(0xffffffffu, v[u].x, other_lane),
                                       __shfl_sync(0xffffffffu, v[u].y, other_lane),
                                       __shfl_sync(0xffffffffu, v[u].z, other_lane),
                                       __shfl_sync(0xffffffffu, v[u].w, other_lane));
          unpack<T>(far, o);
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) o[i] = x[i ^ 1];
        }
        float r[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float own = x[i] * wa[i];
          r[i] = (turns ? fmaf(o[i], wb[i], own) : own) * g;    // an infinite other element of a
                                                                // lane that does not turn stays out
        }
        y = pack<T>(r);
      }
      if (live && (kind == 0 || row >= 0)) *reinterpret_cast<uint4*>(dst + sub * 16) = y;
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
  append_kernel<T, kLanes><<<(unsigned)blocks, kThreads, 0, a.stream>>>(a, (int)per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a) {
  if (a.pv.dtype == KVSEL_BF16)
    return a.pv.D == 128 ? launch<__nv_bfloat16, 16>(a) : launch<__nv_bfloat16, 8>(a);
  return a.pv.D == 128 ? launch<float, 32>(a) : launch<float, 16>(a);
}

}  // namespace kvsel
