// New tokens into a paged cache: per-head norm of queries and keys, position
// rotation, and the rows' places in the pages, in one pass.
//
// Mathematics, per token and head with the row x of D elements:
//   r_i = x_i * rsqrt(mean(x^2) + eps) * w_i                 (r = x without a weight)
//   (y_a, y_b) = scale * (r_a cos t - r_b sin t, r_b cos t + r_a sin t),  t = position * f_i
// for the pairs (a, b) = (i, i + rot/2), or (2i, 2i + 1) when interleaved; the rest of the
// row keeps r. fp32 throughout, one rounding at the store.
//
// Bound by memory: every row is read once and written once.
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

__device__ __forceinline__ void store_elem(char* base, int i, float x, int dtype) {
  if (dtype == KVSEL_BF16)
    reinterpret_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(x);
  else
    reinterpret_cast<float*>(base)[i] = x;
}

// One warp per (layer, token, head); heads 0 .. H-1 are q's, then k's, then v's.
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int hk = a.src[1] ? a.pv.Hkv : 0;
  const int heads = a.H + 2 * hk;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= (int64_t)a.pv.layers * a.tokens * heads) return;
  const int64_t lt = item / heads;
  int h = (int)(item - lt * heads);
  const int layer = (int)(lt / a.tokens), n = (int)(lt - (int64_t)layer * a.tokens);
  const int kind = h < a.H ? 0 : h < a.H + hk ? 1 : 2;
  h -= kind == 0 ? 0 : kind == 1 ? a.H : a.H + hk;
  const int D = a.pv.D, eb = a.pv.dtype == KVSEL_BF16 ? 2 : 4;
  const char* src = a.src[kind] + layer * a.layer_bytes[kind] + n * a.token_bytes[kind] +
                    (int64_t)h * D * eb;
  char* dst;
  if (kind == 0) {
    dst = a.q_out + (((int64_t)layer * a.tokens + n) * a.H + h) * D * eb;
  } else {
    const int pos = a.cache_pos[n];
    if (pos < 0) return;
    int page, r;
    if (!a.table) {
      page = pos >> a.pv.page_shift;
      r = pos & (a.pv.page_size - 1);
      if (page >= a.pv.num_pages) page = -1;
      if (page < 0) record_status(a.status, KVSEL_ERR_BAD_INDEX);
    } else {
      const int b = a.seqs ? a.seqs[n] : n;
      const int col = pos >> a.pv.page_shift;
      r = pos & (a.pv.page_size - 1);
      page = -1;
      if (b >= 0 && b < a.num_seqs && col < a.table_width)
        page = checked_page(a.pv, a.table + (int64_t)b * a.table_width, col, a.status);
      else
        record_status(a.status, KVSEL_ERR_BAD_INDEX);
    }
    if (page < 0) return;
    dst = (kind == 1 ? a.pv.k : a.pv.v) + layer * a.pv.layer_bytes +
          ((int64_t)row_units(a.pv, page, r) + (int64_t)h * a.pv.head_units) * kRowUnit;
  }
  // lane holds elements lane, lane + 32, ..
  float x[4], y[4];
  const int per = D / 32;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = i < per ? load_elem(src, lane + 32 * i, a.pv.dtype) : 0.f;
    ss = fmaf(x[i], x[i], ss);
  }
  if (kind < 2 && a.weight[kind]) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float g = rsqrtf(ss / D + a.eps);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < per) x[i] *= g * load_elem(a.weight[kind], (int64_t)layer * D + lane + 32 * i, a.pv.dtype);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = x[i];
  if (kind < 2 && a.rot > 0) {
    const int half = a.rot / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 32 * i;
      // the partner element's index, and its value from the lane that holds it
      int p = a.interleaved ? e ^ 1 : e < half ? e + half : e - half;
      if (e >= a.rot) p = e;
      float other = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = __shfl_sync(0xffffffffu, x[j], p & 31);
        if ((p >> 5) == j) other = v;
      }
      if (e < a.rot && i < per) {
        const int pair = a.interleaved ? e >> 1 : e < half ? e : e - half;
        const bool first = a.interleaved ? !(e & 1) : e < half;
        float c, s;
        rotation(a.positions[n], a.inv_freq[pair], a.rope_scale, &c, &s);
        y[i] = first ? x[i] * c - other * s : x[i] * c + other * s;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < per) store_elem(dst, lane + 32 * i, y[i], a.pv.dtype);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a) {
  const int heads = a.H + (a.src[1] ? 2 * a.pv.Hkv : 0);
  const int64_t items = (int64_t)a.pv.layers * a.tokens * heads;
  const int64_t blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  append_kernel<<<(unsigned)blocks, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvsel
