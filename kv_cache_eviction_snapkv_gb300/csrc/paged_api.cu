// C entry points of the paged-cache calls: argument rules and descriptors.
// Everything that a step changes (lengths, tables, indices) is read by the
// kernels from device memory, so the calls do no host-to-device copy and no
// allocation and can be captured into a graph.
#include <cmath>

#include "kvsel_internal.h"

namespace kvsel {
namespace {

bool misaligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) & (bytes - 1); }

// The pool's rules (see kvsel.h) and its view. `data`: whether K and V are used.
kvsel_status view_of(const kvsel_pages* p, bool data, PagedView* v) {
  if (!p || p->num_layers < 1 || p->num_pages < 0 || p->page_size < 1 || p->num_kv_heads < 1 ||
      p->head_dim < 1 || (p->dtype != KVSEL_BF16 && p->dtype != KVSEL_F32) ||
      p->layer_stride < 0 || p->page_stride < 0)
    return KVSEL_ERR_INVALID_ARG;
  if ((p->head_dim != 64 && p->head_dim != 128) || (p->page_size & (p->page_size - 1)))
    return KVSEL_ERR_UNSUPPORTED;
  const int eb = p->dtype == KVSEL_BF16 ? 2 : 4;
  const int64_t row = (int64_t)p->num_kv_heads * p->head_dim;
  if ((int64_t)p->num_pages * p->page_size > 0x7fffffffLL || row * eb / kRowUnit > 0x7fffffffLL)
    return KVSEL_ERR_UNSUPPORTED;
  if (row > (int64_t(1) << 40) / p->page_size) return KVSEL_ERR_UNSUPPORTED;
  const int64_t page = row * p->page_size;                     // < 2^40 elements
  const int64_t ps = p->page_stride ? p->page_stride : page;
  if (ps < page || (p->layer_stride && p->layer_stride < page)) return KVSEL_ERR_INVALID_ARG;
  const int64_t per_unit = kRowUnit / eb;
  if (ps % per_unit || p->layer_stride % per_unit) return KVSEL_ERR_INVALID_ARG;
  const int64_t n = p->num_pages > 1 ? p->num_pages - 1 : 1;
  if (ps / per_unit > (0xffffffffLL - page / per_unit) / n) return KVSEL_ERR_UNSUPPORTED;
  const int64_t ls = p->layer_stride ? p->layer_stride : ps * p->num_pages;
  if (ls > (int64_t(1) << 60) / eb / p->num_layers) return KVSEL_ERR_UNSUPPORTED;
  if (data && p->num_pages > 0 &&
      (!p->K || !p->V || misaligned(p->K, kRowUnit) || misaligned(p->V, kRowUnit)))
    return KVSEL_ERR_INVALID_ARG;
  v->k = static_cast<char*>(p->K);
  v->v = static_cast<char*>(p->V);
  v->layer_bytes = ls * eb;
  v->page_units = (uint32_t)(ps / per_unit);
  v->row_units = (uint32_t)(row / per_unit);
  v->head_units = (uint32_t)(p->head_dim / per_unit);
  v->page_size = p->page_size;
  v->page_shift = 0;
  while ((1 << v->page_shift) < p->page_size) ++v->page_shift;
  v->num_pages = p->num_pages;
  v->layers = p->num_layers;
  v->Hkv = p->num_kv_heads;
  v->D = p->head_dim;
  v->dtype = p->dtype;
  return KVSEL_OK;
}

kvsel_status check_table(const PagedView& v, int num_seqs, const int32_t* table, int width) {
  if (num_seqs < 0) return KVSEL_ERR_INVALID_ARG;
  if (num_seqs == 0) return KVSEL_OK;
  if (width < 1 || !table) return KVSEL_ERR_INVALID_ARG;
  // (the kernels' int arithmetic has room above the last row and column)
  if ((int64_t)width * v.page_size >= (int64_t(1) << 30) || (int64_t)num_seqs * width > 0x7fffffffLL)
    return KVSEL_ERR_UNSUPPORTED;
  return KVSEL_OK;
}

}  // namespace
}  // namespace kvsel

using namespace kvsel;

extern "C" {

kvsel_status kvsel_rope_frequencies(int32_t rot_dim, double base, int32_t kind, double factor,
                                    int64_t original_len, double low, double high,
                                    float* inv_freq, float* scale) {
  if (rot_dim < 2 || rot_dim % 2 || !(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) ||
      !std::isfinite(factor) || kind < KVSEL_ROPE_PLAIN || kind > KVSEL_ROPE_PARTS || !inv_freq ||
      !scale)
    return KVSEL_ERR_INVALID_ARG;
  if (kind == KVSEL_ROPE_BASE) {
    if (rot_dim == 2) return KVSEL_ERR_INVALID_ARG;
    base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  }
  if (kind == KVSEL_ROPE_PARTS && (original_len < 1 || !(low > 0.0) || !(high > low)))
    return KVSEL_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (kind == KVSEL_ROPE_LINEAR) f /= factor;
    if (kind == KVSEL_ROPE_PARTS) {
      // turns over the original context: few -> stretched, many -> left
      const double turns = (double)original_len * f / 6.283185307179586;
      double keep = (turns - low) / (high - low);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f = f * keep + f / factor * (1.0 - keep);
    }
    inv_freq[i] = (float)f;
  }
  *scale = kind == KVSEL_ROPE_PARTS ? (float)(1.0 + 0.1 * std::log(factor)) : 1.0f;
  return KVSEL_OK;
}

kvsel_status kvsel_paged_append(const kvsel_pages* pages, int32_t num_tokens, int32_t num_heads,
                                const kvsel_rows* q, const kvsel_rows* k, const kvsel_rows* v,
                                const kvsel_rope* rope, const void* q_weight,
                                const void* k_weight, float eps, const int32_t* positions,
                                int32_t num_seqs, const int32_t* table, int32_t table_width,
                                const int32_t* seqs, const int32_t* cache_pos, void* q_out,
                                void* stream) {
  AppendArgs a{};
  kvsel_status st;
  if ((st = view_of(pages, k != nullptr, &a.pv))) return st;
  if (num_tokens < 0 || num_heads < (q ? 1 : 0) || !(eps >= 0.f) || !std::isfinite(eps) ||
      (k == nullptr) != (v == nullptr))
    return KVSEL_ERR_INVALID_ARG;
  const int rot = rope ? rope->rot_dim : 0;
  if (rot < 0 || (rot > 0 && !std::isfinite(rope->scale))) return KVSEL_ERR_INVALID_ARG;
  if (rot > a.pv.D || rot % 16) return KVSEL_ERR_UNSUPPORTED;
  const int64_t heads = (int64_t)num_heads + 2 * (int64_t)a.pv.Hkv;
  if (heads > 65535 || (double)a.pv.layers * num_tokens * (double)heads >= 4294967296.0)
    return KVSEL_ERR_UNSUPPORTED;
  if (k && table) {
    if ((st = check_table(a.pv, num_seqs, table, table_width))) return st;
    if (!seqs && num_tokens > num_seqs) return KVSEL_ERR_INVALID_ARG;
  }
  if (num_tokens == 0 || (!q && !k)) return KVSEL_OK;
  if (rot > 0 && (!rope->inv_freq || !positions)) return KVSEL_ERR_INVALID_ARG;
  if ((q && !q_out) || (k && !cache_pos)) return KVSEL_ERR_INVALID_ARG;
  if (misaligned(q_weight, 16) || misaligned(k_weight, 16) || misaligned(q_out, 16))
    return KVSEL_ERR_INVALID_ARG;
  const int eb = a.pv.dtype == KVSEL_BF16 ? 2 : 4;
  const kvsel_rows* rows[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    if (!rows[i]) continue;
    const kvsel_rows& r = *rows[i];
    if (!r.data || misaligned(r.data, 16) || r.layer_stride < 0 || r.token_stride < 0 ||
        (r.layer_stride * eb) % 16 || (r.token_stride * eb) % 16)
      return KVSEL_ERR_INVALID_ARG;
    a.src[i] = static_cast<const char*>(r.data);
    a.layer_bytes[i] = r.layer_stride * eb;
    a.token_bytes[i] = r.token_stride * eb;
  }
  DeviceInfo d;
  if ((st = device_info(&d))) return st;
  a.q_out = static_cast<char*>(q_out);
  a.tokens = num_tokens;
  a.H = q ? num_heads : 0;
  a.rot = rot;
  if (rot > 0) {
    a.interleaved = rope->interleaved != 0;
    a.inv_freq = rope->inv_freq;
    a.rope_scale = rope->scale;
  }
  a.weight[0] = static_cast<const char*>(q_weight);
  a.weight[1] = static_cast<const char*>(k_weight);
  a.eps = eps;
  a.positions = positions;
  a.table = table;
  a.table_width = table_width;
  a.num_seqs = num_seqs;
  a.seqs = seqs;
  a.cache_pos = cache_pos;
  a.status = d.status;
  a.sm_count = d.sm_count;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_append(a), "paged append launch");
}

static kvsel_status attention_view(const kvsel_pages* pages, bool data, int32_t num_seqs,
                                   int32_t num_heads, PagedView* v) {
  const kvsel_status st = view_of(pages, data, v);
  if (st) return st;
  if (num_seqs < 0 || num_heads < 1 || num_heads % v->Hkv) return KVSEL_ERR_INVALID_ARG;
  if (num_seqs > kMaxPagedSeqs ||
      (double)v->layers * num_seqs * num_heads > 2147483647.0)
    return KVSEL_ERR_UNSUPPORTED;
  return KVSEL_OK;
}

int64_t kvsel_paged_attention_bytes(const kvsel_pages* pages, int32_t num_seqs,
                                    int32_t num_heads) {
  PagedView v;
  DeviceInfo d;
  if (attention_view(pages, false, num_seqs, num_heads, &v) || device_info(&d)) return -1;
  return paged_attention_ws(v, num_seqs, num_heads, d.sm_count);
}

kvsel_status kvsel_paged_attention(const kvsel_pages* pages, int32_t num_seqs, int32_t num_heads,
                                   const void* q, const int32_t* table, int32_t table_width,
                                   const int32_t* lens, float* out, float* lse, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  PagedAttnArgs a{};
  kvsel_status st;
  if ((st = attention_view(pages, true, num_seqs, num_heads, &a.pv))) return st;
  if ((st = check_table(a.pv, num_seqs, table, table_width))) return st;
  if (num_seqs == 0) return KVSEL_OK;
  if ((int64_t)num_seqs * table_width > (int64_t(1) << 34) / a.pv.page_size)
    return KVSEL_ERR_UNSUPPORTED;
  if (!q || !lens || !out || misaligned(q, 16) || misaligned(out, 16))
    return KVSEL_ERR_INVALID_ARG;
  DeviceInfo d;
  if ((st = device_info(&d))) return st;
  const int64_t need = paged_attention_ws(a.pv, num_seqs, num_heads, d.sm_count);
  if (workspace_bytes < need || (need > 0 && (!workspace || misaligned(workspace, 16))))
    return KVSEL_ERR_INVALID_ARG;
  a.q = q;
  a.table = table;
  a.table_width = table_width;
  a.lens = lens;
  a.S = num_seqs;
  a.H = num_heads;
  a.out = out;
  a.lse = lse;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)a.pv.D));
  a.ws = static_cast<char*>(workspace);
  a.status = d.status;
  a.sm_count = d.sm_count;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_paged_attention(a), "paged attention launch");
}

kvsel_status kvsel_paged_compact(const kvsel_pages* pages, int32_t num_seqs, const int32_t* table,
                                 int32_t table_width, const int32_t* lens,
                                 const int32_t* keep_idx, int64_t keep_rows,
                                 const int32_t* keep_offsets, int32_t max_keep,
                                 const int32_t* ref, int32_t* slot_pos, void* stream) {
  PagedCompactArgs a{};
  kvsel_status st;
  if ((st = view_of(pages, true, &a.pv))) return st;
  if ((st = check_table(a.pv, num_seqs, table, table_width))) return st;
  if (max_keep < 0 || keep_rows < 0) return KVSEL_ERR_INVALID_ARG;
  if (max_keep > kMaxKeep || (double)a.pv.layers * num_seqs * a.pv.Hkv > 2147483647.0 ||
      keep_rows > 0x7fffffffLL)
    return KVSEL_ERR_UNSUPPORTED;
  if (num_seqs == 0 || keep_rows == 0 || max_keep == 0) return KVSEL_OK;
  if (!lens || !keep_idx || !keep_offsets) return KVSEL_ERR_INVALID_ARG;
  DeviceInfo d;
  if ((st = device_info(&d))) return st;
  a.table = table;
  a.table_width = table_width;
  a.S = num_seqs;
  a.lens = lens;
  a.keep_idx = keep_idx;
  a.keep_rows = keep_rows;
  a.keep_offsets = keep_offsets;
  a.max_keep = max_keep;
  a.ref = ref;
  a.slot_pos = slot_pos;
  a.status = d.status;
  a.sm_count = d.sm_count;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_paged_compact(a), "paged compaction launch");
}

int64_t kvsel_pages_update_bytes(const kvsel_pages* pages, int32_t num_out) {
  PagedView v;
  if (view_of(pages, false, &v) || num_out < 0) return -1;
  return pages_update_ws(v.num_pages, num_out);
}

kvsel_status kvsel_pages_update(const kvsel_pages* pages, int32_t num_in, const int32_t* table,
                                int32_t table_width, const int32_t* lens, int32_t num_out,
                                const int32_t* parents, const int32_t* new_lens,
                                int32_t* table_out, int32_t* ref, int32_t* free_pages,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  PagesUpdateArgs a{};
  kvsel_status st;
  if ((st = view_of(pages, true, &a.pv))) return st;
  if ((st = check_table(a.pv, num_in, table, table_width))) return st;
  if ((st = check_table(a.pv, num_out, table_out, table_width))) return st;
  if ((num_in > 0 && !lens) || (num_out > 0 && !new_lens) || (a.pv.num_pages > 0 && !ref) ||
      (!parents && num_out > 0 && num_in != num_out))
    return KVSEL_ERR_INVALID_ARG;
  if (num_in > 0 && num_out > 0) {
    const int32_t* in_end = table + (int64_t)num_in * table_width;
    const int32_t* out_end = table_out + (int64_t)num_out * table_width;
    if (table < out_end && table_out < in_end) return KVSEL_ERR_INVALID_ARG;
  }
  const int64_t need = pages_update_ws(a.pv.num_pages, num_out);
  if (workspace_bytes < need || !workspace || misaligned(workspace, 16))
    return KVSEL_ERR_INVALID_ARG;
  DeviceInfo d;
  if ((st = device_info(&d))) return st;
  a.num_in = num_in;
  a.num_out = num_out;
  a.table_width = table_width;
  a.table = table;
  a.lens = lens;
  a.parents = parents;
  a.new_lens = new_lens;
  a.table_out = table_out;
  a.ref = ref;
  a.free_pages = free_pages;
  a.ws = static_cast<char*>(workspace);
  a.status = d.status;
  a.sm_count = d.sm_count;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_pages_update(a), "pages update launch");
}

}  // extern "C"
