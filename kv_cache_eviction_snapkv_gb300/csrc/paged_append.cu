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
// neighbours. An element then costs a product and a sum, two elements at a time (the fp32 pair
// instructions), and no exchange between lanes but the norm's sum. (With 16 contiguous bytes a
// lane and the other half fetched by shuffles, 16384 tokens took 105 us, 74% of the issue slots
// used.) The loads go through a ring of shared memory, seven passes ahead without a register:
// every lane copies what it will read itself, so nothing but its own copies is waited for.
//
// Measured: 16384 tokens of 32 + 8 + 8 heads of 128 in bf16, 403 MB: 71 us, 5.7 TB/s, 84% of the
// copy bandwidth; 16 tokens: 3.4 us.
#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 128;   // small blocks: the last ones leave less of the machine idle

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

// 16 bytes of a row: eight bf16 or four fp32 values, in twos.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, Two (&x)[8 / sizeof(T)]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8 / (int)sizeof(T); ++i) {
    if constexpr (sizeof(T) == 2)
      x[i] = two(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else
      x[i] = two(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const Two (&x)[8 / sizeof(T)]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 8 / (int)sizeof(T); ++i) {
    const float2 f = both(x[i]);
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      w[2 * i] = __float_as_uint(f.x);
      w[2 * i + 1] = __float_as_uint(f.y);
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
__global__ void __launch_bounds__(kThreads, 7) append_kernel(const __grid_constant__ AppendArgs a,
                                                             int per_warp) {
  constexpr int N = 8 / sizeof(T), U = N;         // twos of a lane, its pairs
  constexpr int D = kLanes * 2 * N, kHeads = 32 / kLanes, kRowBytes = kLanes * 16;
  constexpr int kRing = 8;                        // passes in the ring
  constexpr int kSlot = kThreads * 16;
  __shared__ __align__(16) unsigned char ring[kRing][kSlot];
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
  const bool turns = sub < a.rot / (2 * N);
  const bool apart = !kInterleaved && turns;
  const int ua = (apart ? sub : 2 * sub) * 8;     // byte offsets
  const int ub = apart ? ua + a.rot / 2 * (int)sizeof(T) : ua + 8;

  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(&ring[0][threadIdx.x * 16]);
  // the heads of passes [b, e) of a kind that this lane's group has, and the first one's place
  auto heads_of = [&](int b, int e, int heads) {
    const int h = (heads - b * kHeads - grp + kHeads - 1) / kHeads;
    return max(0, min(e - b, h));
  };
  const char* src = nullptr;
  int left = 0;
  uint32_t in = mine;
  auto issue = [&] {
    if (left > 0) {
      copy8(in, src + ua);
      copy8(in + 8, src + ub);
    }
    src += kHeads * kRowBytes;
    --left;
    in = in == mine + (kRing - 1) * kSlot ? mine : in + kSlot;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto begin = [&](int kind, int b, int e) {
    src = a.src[kind] + layer * a.layer_bytes[kind] + n * a.token_bytes[kind] +
          (b * kHeads + grp) * kRowBytes;
    left = heads_of(b, e, kind == 0 ? a.H : hk);
    in = mine;
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) issue();
  };

  const int q0 = min(p0, pq), q1 = min(p1, pq);
  const int k0 = min(max(p0 - pq, 0), pk), k1 = min(max(p1 - pq, 0), pk);
  const int v0 = min(max(p0 - pq - pk, 0), pk), v1 = min(max(p1 - pq - pk, 0), pk);
  if (q0 < q1) begin(0, q0, q1);
  else if (k0 < k1) begin(1, k0, k1);
  const int64_t row = p1 > pq ? target_row(a, n) : -1;

  float c[U], s[U];                               // of this lane's pairs
  const bool rotates = turns && p0 < pq + pk;
  if (rotates) {
    const int position = a.positions[n];
#pragma unroll
    for (int i = 0; i < U; ++i)
      rotation(position, a.inv_freq[sub * U + i], a.rope_scale, &c[i], &s[i]);
  }
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const int b = kind == 0 ? q0 : k0, e = kind == 0 ? q1 : k1;
    if (b >= e) continue;
    if (kind == 1 && q0 < q1) begin(1, k0, k1);
    char* dst = kind == 0 ? a.q_out + ((int64_t)layer * a.tokens + n) * a.H * kRowBytes
                          : a.pv.k + layer * a.pv.layer_bytes + row;
    dst += (int64_t)(b * kHeads + grp) * kRowBytes;
    int out = kind == 0 || row >= 0 ? heads_of(b, e, kind == 0 ? a.H : hk) : 0;
    const char* weight = kind == 0 ? a.weight[0] : a.weight[1];
    // twos v, with w the other elements of their pairs, become (v va + w vb) g: cosines and
    // sines times weights
    Two va[N], vb[N];
    {
      Two w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = two(1.f, 1.f);
      if (weight) {
        const char* at = weight + (int64_t)layer * kRowBytes;
        const uint2 x = *reinterpret_cast<const uint2*>(at + ua), y = *reinterpret_cast<const uint2*>(at + ub);
        unpack<T>(make_uint4(x.x, x.y, y.x, y.y), w);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        va[i] = w[i];
        vb[i] = two(0.f, 0.f);
        if (!rotates) continue;
        if (kInterleaved) {
          const float2 f = both(w[i]);
          va[i] = mul(w[i], two(c[i], c[i]));
          vb[i] = two(-f.y * s[i], f.x * s[i]);
        } else {
          const int j = 2 * (i % (N / 2));
          const float sign = i < N / 2 ? -1.f : 1.f;
          va[i] = mul(w[i], two(c[j], c[j + 1]));
          vb[i] = mul(w[i ^ (N / 2)], two(sign * s[j], sign * s[j + 1]));
        }
      }
    }
    uint32_t at = mine;
#pragma unroll 2
    for (int p = b; p < e; ++p) {
      issue();                                    // into the slot that was read a pass ago
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      const uint4 raw = shared16(at);
      at = at == mine + (kRing - 1) * kSlot ? mine : at + kSlot;
      Two x[N], r[N];
      unpack<T>(raw, x);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        r[i] = mul(x[i], va[i]);
        if (turns) {                              // elsewhere an infinite neighbour must stay out
          const float2 f = both(x[i]);
          r[i] = fma(kInterleaved ? two(f.y, f.x) : x[i ^ (N / 2)], vb[i], r[i]);
        }
      }
      if (weight) {
        Two ss = mul(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < N; ++i) ss = fma(x[i], x[i], ss);
        const float2 f = both(ss);
        float sum = f.x + f.y;
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const float g = rsqrtf(fmaf(sum, 1.f / D, a.eps));
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = mul(r[i], two(g, g));
      }
      const uint4 y = pack<T>(r);
      if (out > 0) {
        *reinterpret_cast<uint2*>(dst + ua) = make_uint2(y.x, y.y);
        *reinterpret_cast<uint2*>(dst + ub) = make_uint2(y.z, y.w);
      }
      dst += kHeads * kRowBytes;
      --out;
    }
  }
  // v, as it is
  if (v0 < v1 && row >= 0) {
    const int64_t first = (int64_t)(v0 * kHeads + grp) * kRowBytes + sub * 16;
    const char* from = a.src[2] + layer * a.layer_bytes[2] + n * a.token_bytes[2] + first;
    char* to = a.pv.v + layer * a.pv.layer_bytes + row + first;
    const int heads = heads_of(v0, v1, hk);
    for (int i0 = 0; i0 < heads; i0 += 4) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i < heads)
          v[i] = __ldcs(reinterpret_cast<const uint4*>(from + (i0 + i) * (kHeads * kRowBytes)));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i < heads) *reinterpret_cast<uint4*>(to + (i0 + i) * (kHeads * kRowBytes)) = v[i];
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
