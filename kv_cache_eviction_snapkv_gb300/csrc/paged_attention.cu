// One new query per (layer, sequence, query head) over a paged cache.
//
// Mathematics: s_j = q . k_j / sqrt(D) over the rows j < len, running maximum m and sum l of
// exp(s - m), out = sum_j exp(s_j - m) v_j / l, lse = m + ln l; an empty sequence has out = 0
// and lse = -inf. Everything in fp32, in base-2 units until the end.
#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// One block per (layer, sequence, query head); its warps take rows in turn, a lane holds D/32
// elements.
__global__ void __launch_bounds__(kThreads) paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  __shared__ float wm[kWarps], wl[kWarps], wo[kWarps][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t inst = blockIdx.x;
  const int h = (int)(inst % a.H);
  const int b = (int)(inst / a.H % a.S), layer = (int)(inst / a.H / a.S);
  const int kvh = h / (a.H / a.pv.Hkv);
  const int D = a.pv.D, per = D / 32;
  const int len = checked_len(a.lens[b], a.table_width << a.pv.page_shift, a.status);
  const int32_t* trow = a.table + (int64_t)b * a.table_width;
  const int64_t base = layer * a.pv.layer_bytes + (int64_t)kvh * a.pv.head_units * kRowUnit;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = i < per ? load_elem(a.q, inst * D + lane * per + i, a.pv.dtype) * a.scale_log2 : 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < len; j += kWarps) {
    const int page = checked_page(a.pv, trow, j >> a.pv.page_shift, a.status);
    if (page < 0) continue;
    const int64_t off = base + (int64_t)row_units(a.pv, page, j & (a.pv.page_size - 1)) * kRowUnit;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < per) s = fmaf(q[i], load_elem(a.pv.k + off, lane * per + i, a.pv.dtype), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mx = fmaxf(m, s);
    const float f = mx == -INFINITY ? 1.f : ex2(m - mx);
    const float p = s == -INFINITY ? 0.f : ex2(s - mx);   // NaN stays NaN
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < per) o[i] = fmaf(p, load_elem(a.pv.v + off, lane * per + i, a.pv.dtype), o[i] * f);
    m = mx;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < per) wo[warp][lane * per + i] = o[i];
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
  __syncthreads();
  float mx = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, wm[w]);
  for (int w = 0; w < kWarps; ++w) sum = fmaf(wl[w], wm[w] == -INFINITY ? 0.f : ex2(wm[w] - mx), sum);
  bool bad = !finite_f(sum) || (sum > 0.f && !finite_f(mx));
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float acc = 0.f;
    for (int w = 0; w < kWarps; ++w)
      acc = fmaf(wo[w][d], wm[w] == -INFINITY ? 0.f : ex2(wm[w] - mx), acc);
    const float v = sum == 0.f ? 0.f : acc / sum;
    bad |= !finite_f(v);
    a.out[inst * D + d] = v;
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[inst] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
  if (bad) record_status(a.status, KVSEL_ERR_NONFINITE);
}

}  // namespace

int64_t paged_attention_ws(const PagedView&, int, int, int) { return 0; }

cudaError_t launch_paged_attention(const PagedAttnArgs& a) {
  const int64_t insts = (int64_t)a.pv.layers * a.S * a.H;
  paged_attn_kernel<<<(unsigned)insts, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvsel
