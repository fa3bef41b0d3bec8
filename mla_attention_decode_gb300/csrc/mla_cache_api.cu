// mla_cache_api.cu -- entry points of the cache operators: argument validation
// and launches (include/mla_cache.h).
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "mla_cache.h"
#include "mla_cache_internal.h"

namespace {

constexpr int32_t kMaxTokens = 1 << 27;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_cache(const mla_cache* c) {
  if (!c) return MLA_ERR_INVALID_ARG;
  if (c->kv_dtype < MLA_KV_BF16 || c->kv_dtype > MLA_KV_MXFP4) return MLA_ERR_UNSUPPORTED;
  if (c->page_size < 1 || c->page_size > (1 << 20) || (c->page_size & (c->page_size - 1)) != 0)
    return MLA_ERR_UNSUPPORTED;
  if (c->num_pages < 0 || c->num_layers < 1 || c->reserved != 0 || c->reserved2 != 0) return MLA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)c->num_pages * c->page_size;
  if (rows > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  if ((rows > 0 && !c->kv) || !aligned(c->kv, 16)) return MLA_ERR_INVALID_ARG;
  if (c->num_layers > 1 &&
      (c->kv_layer_bytes % 16 != 0 || c->kv_layer_bytes < rows * mla::cache_row_bytes(c->kv_dtype)))
    return MLA_ERR_INVALID_ARG;
  if (c->scale_width != 0 && (c->kv_dtype != MLA_KV_MXFP4 || c->scale_width < MLA_MX_SCALES_PER_ROW ||
                              c->scale_width > c->scale_stride))
    return MLA_ERR_INVALID_ARG;
  if (c->kv_dtype == MLA_KV_FP8_E4M3) {
    if (!c->kv_scale || !aligned(c->kv_scale, 4)) return MLA_ERR_INVALID_ARG;
    if (c->num_layers > 1 && (c->scale_layer_bytes < 0 || c->scale_layer_bytes % 4 != 0)) return MLA_ERR_INVALID_ARG;
  } else if (c->kv_dtype == MLA_KV_MXFP4) {
    if ((rows > 0 && !c->kv_scale) || !aligned(c->kv_scale, 16) || c->scale_stride < MLA_MX_SCALES_PER_ROW)
      return MLA_ERR_INVALID_ARG;
    if (c->num_layers > 1 && c->scale_layer_bytes < rows * c->scale_stride) return MLA_ERR_INVALID_ARG;
  }
  return MLA_OK;
}

mla::LayerRows layer_rows(const mla_cache* c, int32_t layer) {
  mla::LayerRows r;
  // one layer: the layer strides are not read
  r.kv = static_cast<uint8_t*>(c->kv) + (layer ? layer * c->kv_layer_bytes : 0);
  r.scale = c->kv_dtype == MLA_KV_BF16
                ? nullptr
                : static_cast<void*>(static_cast<uint8_t*>(c->kv_scale) + (layer ? layer * c->scale_layer_bytes : 0));
  r.scale_stride = c->kv_dtype == MLA_KV_MXFP4 ? c->scale_stride : 0;
  r.rows = c->num_pages * c->page_size;
  return r;
}

int log2_of(int32_t p) {
  int s = 0;
  while ((1 << s) < p) ++s;
  return s;
}

// `rows_moved`: the scale rows that move together at least (1, or a whole page).
mla::PageBytes page_bytes(const mla_cache* c, int32_t rows_moved) {
  mla::PageBytes b;
  std::memset(&b, 0, sizeof b);
  b.kv = static_cast<uint8_t*>(c->kv);
  b.kv_layer = c->num_layers > 1 ? c->kv_layer_bytes : 0;
  b.row_bytes = mla::cache_row_bytes(c->kv_dtype);
  b.page_size = c->page_size;
  b.page_shift = log2_of(c->page_size);
  b.num_pages = c->num_pages;
  b.num_layers = c->num_layers;
  b.scale_unit = 16;
  if (c->kv_dtype == MLA_KV_MXFP4) {
    const bool whole = c->scale_width == 0 || c->scale_width == c->scale_stride;
    (whole ? b.scale : b.scale_cols) = static_cast<uint8_t*>(c->kv_scale);
    b.scale_layer = c->num_layers > 1 ? c->scale_layer_bytes : 0;
    b.scale_stride = c->scale_stride;
    b.scale_width = whole ? c->scale_stride : c->scale_width;
    // every address and length of the call: runs of whole rows, or single rows' columns
    const int64_t step = (int64_t)c->scale_stride * (whole ? rows_moved : 1), len = whole ? step : c->scale_width;
    while (step % b.scale_unit != 0 || len % b.scale_unit != 0 || b.scale_layer % b.scale_unit != 0) b.scale_unit /= 2;
  }
  return b;
}

int check_table(const mla_page_table* t) {
  if (!t || t->batch < 0 || t->batch > MLA_MAX_BATCH || t->num_indices < 0) return MLA_ERR_INVALID_ARG;
  if (!t->page_indptr || !aligned(t->page_indptr, 4) || !aligned(t->kv_indices, 4) || !aligned(t->last_page_len, 4))
    return MLA_ERR_INVALID_ARG;
  if ((t->num_indices > 0 && !t->kv_indices) || (t->batch > 0 && !t->last_page_len)) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

bool multiple(int64_t stride, int64_t of) { return stride % of == 0; }

int done(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  cudaGetLastError();
  return MLA_ERR_CUDA;
}

int table_call(const mla_cache* cache, int32_t* page_refs, const mla_page_table* from, const int32_t* by, bool forks,
               const mla_page_table* to, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_cache(cache);
  if (rc == MLA_OK) rc = check_table(from);
  if (rc == MLA_OK) rc = check_table(to);
  if (rc != MLA_OK) return rc;
  if (to->batch > 0 && (!by || !aligned(by, 4))) return MLA_ERR_INVALID_ARG;
  if (from->page_indptr == to->page_indptr || (from->kv_indices && from->kv_indices == to->kv_indices) ||
      (from->last_page_len && from->last_page_len == to->last_page_len))
    return MLA_ERR_INVALID_ARG;
  if ((cache->num_pages > 0 && !page_refs) || !aligned(page_refs, 16)) return MLA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  mla::TableParams p;
  p.ws = mla::page_ws(workspace, cache->num_pages, to->batch);
  if (workspace_bytes < p.ws.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  p.c = page_bytes(cache, 1);
  p.refs = page_refs;
  p.from = *from;
  p.to = *to;
  p.by = by;
  p.forks = forks;
  p.entries_apart = 0;
  return done(mla::launch_table(p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int mla_rope_plan(const double* inv_freq, const int32_t* axis_of_pair, int32_t num_axes, int32_t interleaved,
                  double scale, mla_rope* rope) {
  if (!inv_freq || !rope || num_axes < 1 || num_axes > MLA_MAX_AXES || (interleaved != 0 && interleaved != 1))
    return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite((float)scale)) return MLA_ERR_INVALID_ARG;
  mla_rope r;
  std::memset(&r, 0, sizeof r);
  for (int i = 0; i < MLA_PE_PAIRS; ++i) {
    if (!std::isfinite(inv_freq[i])) return MLA_ERR_INVALID_ARG;
    const int32_t a = axis_of_pair ? axis_of_pair[i] : 0;
    if (a < 0 || a >= num_axes) return MLA_ERR_INVALID_ARG;
    r.axis[i] = static_cast<uint8_t>(a);
    // the fraction of a turn as a multiple of 2^-64 (2^64 itself is 0 turns); a negative
    // one as that many less than 2^64 (1 less the fraction would round it to 2^-54)
    const double f = std::fmod(std::fabs(inv_freq[i]) / 6.283185307179586476925286766559, 1.0);
    const double u = std::nearbyint(std::ldexp(f, 64));
    const uint64_t turn = u >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(u);
    r.turn[i] = inv_freq[i] < 0 ? 0 - turn : turn;
  }
  r.num_axes = num_axes;
  r.interleaved = interleaved;
  r.scale = static_cast<float>(scale);
  *rope = r;
  return MLA_OK;
}

int mla_cache_append(const mla_cache* cache, const mla_rope* rope, const mla_norm* norm, const mla_append_args* args,
                     int32_t* device_error, void* stream) {
  int rc = check_cache(cache);
  if (rc != MLA_OK) return rc;
  if (!args || args->num_tokens < 0 || args->num_tokens > kMaxTokens) return MLA_ERR_INVALID_ARG;
  if (args->layer < 0 || args->layer >= cache->num_layers || !aligned(device_error, 4)) return MLA_ERR_INVALID_ARG;
  mla::AppendParams p;
  std::memset(&p, 0, sizeof p);
  if (rope) {
    if (rope->num_axes < 1 || rope->num_axes > MLA_MAX_AXES || !std::isfinite(rope->scale)) return MLA_ERR_INVALID_ARG;
    for (int i = 0; i < MLA_PE_PAIRS; ++i)
      if (rope->axis[i] >= rope->num_axes) return MLA_ERR_INVALID_ARG;
    p.rope = *rope;
  }
  if (norm) {
    if ((norm->apply & ~15) != 0 || (norm->weight_fp32 != 0 && norm->weight_fp32 != 1)) return MLA_ERR_INVALID_ARG;
    if (!std::isfinite(norm->eps) || norm->eps < 0) return MLA_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i)
      if (!aligned(norm->weight[i], 16)) return MLA_ERR_INVALID_ARG;
    p.norm = *norm;
  }
  if (args->num_tokens == 0) return MLA_OK;
  const mla_append_args& a = *args;
  if (a.kv_lat) {
    if (!a.kv_pe || !a.slots || !aligned(a.slots, 4)) return MLA_ERR_INVALID_ARG;
    if (!aligned(a.kv_lat, 16) || !aligned(a.kv_pe, 4)) return MLA_ERR_INVALID_ARG;
    if (!multiple(a.kv_lat_stride, 8) || !multiple(a.kv_pe_stride, 2)) return MLA_ERR_INVALID_ARG;
  } else if (a.kv_pe) {
    return MLA_ERR_INVALID_ARG;
  }
  if (a.q_pe) {
    if (!a.q_out || !aligned(a.q_pe, 4) || !aligned(a.q_out, 16) || !aligned(a.q_lat, 16)) return MLA_ERR_INVALID_ARG;
    if (!multiple(a.q_pe_token_stride, 2) || !multiple(a.q_pe_head_stride, 2)) return MLA_ERR_INVALID_ARG;
    if (a.q_lat && (!multiple(a.q_lat_token_stride, 8) || !multiple(a.q_lat_head_stride, 8)))
      return MLA_ERR_INVALID_ARG;
  } else if (a.q_lat || a.q_out) {
    return MLA_ERR_INVALID_ARG;
  }
  if (rope && (!a.positions || !aligned(a.positions, 4))) return MLA_ERR_INVALID_ARG;
  p.cache = layer_rows(cache, args->layer);
  p.a = a;
  p.error = device_error;
  return done(mla::launch_append(p, cache->kv_dtype, static_cast<cudaStream_t>(stream)));
}

int mla_cache_gather(const mla_cache* cache, int32_t layer, const int32_t* slots, int32_t num_rows, void* out,
                     int64_t out_stride, int32_t* device_error, void* stream) {
  const int rc = check_cache(cache);
  if (rc != MLA_OK) return rc;
  if (layer < 0 || layer >= cache->num_layers || num_rows < 0 || num_rows > kMaxTokens || !aligned(device_error, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_rows == 0) return MLA_OK;
  if (!slots || !out || !aligned(slots, 4) || !aligned(out, 16)) return MLA_ERR_INVALID_ARG;
  if (out_stride < mla::kRow || !multiple(out_stride, 8)) return MLA_ERR_INVALID_ARG;
  mla::GatherParams p;
  p.cache = layer_rows(cache, layer);
  p.slots = slots;
  p.out = static_cast<uint8_t*>(out);
  p.out_stride = out_stride * 2;
  p.num_rows = num_rows;
  p.error = device_error;
  return done(mla::launch_gather(p, cache->kv_dtype, static_cast<cudaStream_t>(stream)));
}

int mla_cache_slots(const mla_cache* cache, const mla_page_table* table, const int32_t* qo_indptr, int32_t num_tokens,
                    int32_t* slots, int32_t* rows, int64_t row_stride, int32_t* device_error, void* stream) {
  int rc = check_cache(cache);
  if (rc == MLA_OK) rc = check_table(table);
  if (rc != MLA_OK) return rc;
  if (num_tokens < 0 || num_tokens > kMaxTokens || !aligned(device_error, 4)) return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (!qo_indptr || !slots || !aligned(qo_indptr, 4) || !aligned(slots, 4) || !aligned(rows, 4))
    return MLA_ERR_INVALID_ARG;
  mla::SlotsParams p;
  p.table = *table;
  p.qo_indptr = qo_indptr;
  p.slots = slots;
  p.rows = rows;
  p.row_stride = row_stride;
  p.num_tokens = num_tokens;
  p.page_shift = log2_of(cache->page_size);
  p.num_pages = cache->num_pages;
  p.error = device_error;
  return done(mla::launch_slots(p, static_cast<cudaStream_t>(stream)));
}

int mla_cache_copy_pages(const mla_cache* cache, const int32_t* src, const int32_t* dst, int32_t n,
                         int32_t* device_error, void* stream) {
  const int rc = check_cache(cache);
  if (rc != MLA_OK) return rc;
  if (n < 0 || !aligned(device_error, 4)) return MLA_ERR_INVALID_ARG;
  if (n == 0) return MLA_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return MLA_ERR_INVALID_ARG;
  mla::CopyParams p;
  p.c = page_bytes(cache, cache->page_size);
  p.src = src;
  p.dst = dst;
  p.n = n;
  p.error = device_error;
  return done(mla::launch_copy_pages(p, static_cast<cudaStream_t>(stream)));
}

int mla_cache_fork(const mla_cache* cache, int32_t* page_refs, const mla_page_table* from, const int32_t* parents,
                   const mla_page_table* to, void* workspace, size_t workspace_bytes, void* stream) {
  return table_call(cache, page_refs, from, parents, true, to, workspace, workspace_bytes, stream);
}

int mla_cache_resize(const mla_cache* cache, int32_t* page_refs, const mla_page_table* from, const int32_t* lengths,
                     const mla_page_table* to, void* workspace, size_t workspace_bytes, void* stream) {
  if (!from || !to || from->batch != to->batch) return MLA_ERR_INVALID_ARG;
  return table_call(cache, page_refs, from, lengths, false, to, workspace, workspace_bytes, stream);
}

int mla_cache_free(const mla_cache* cache, int32_t* page_refs, const int32_t* pages, int32_t n, int32_t* device_error,
                   void* stream) {
  const int rc = check_cache(cache);
  if (rc != MLA_OK) return rc;
  if (n < 0 || !aligned(device_error, 4)) return MLA_ERR_INVALID_ARG;
  if (n == 0) return MLA_OK;
  if (!pages || !aligned(pages, 4) || (cache->num_pages > 0 && !page_refs) || !aligned(page_refs, 16))
    return MLA_ERR_INVALID_ARG;
  return done(mla::launch_free(page_refs, cache->num_pages, pages, n, device_error, static_cast<cudaStream_t>(stream)));
}

int mla_cache_compact(const mla_cache* cache, const int32_t* page_refs, int32_t* page_refs_out,
                      const int32_t* kv_indices, int32_t* kv_indices_out, int32_t num_indices, int32_t* live,
                      void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_cache(cache);
  if (rc != MLA_OK) return rc;
  if (num_indices < 0 || !aligned(live, 4)) return MLA_ERR_INVALID_ARG;
  if ((cache->num_pages > 0 && (!page_refs || !page_refs_out)) || !aligned(page_refs, 16) || !aligned(page_refs_out, 16))
    return MLA_ERR_INVALID_ARG;
  if (num_indices > 0 && (!kv_indices || !kv_indices_out || !aligned(kv_indices, 4) || !aligned(kv_indices_out, 4)))
    return MLA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  mla::CompactParams p;
  p.ws = mla::page_ws(workspace, cache->num_pages, 0);
  if (workspace_bytes < p.ws.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  p.c = page_bytes(cache, cache->page_size);
  p.refs_in = page_refs;
  p.refs_out = page_refs_out;
  p.idx_in = kv_indices;
  p.idx_out = kv_indices_out;
  p.num_indices = num_indices;
  p.live = live;
  p.entries_apart = 0;
  return done(mla::launch_compact(p, static_cast<cudaStream_t>(stream)));
}

size_t mla_cache_workspace_bytes(const mla_cache* cache, int32_t batch) {
  if (check_cache(cache) != MLA_OK || batch < 0 || batch > MLA_MAX_BATCH) return 0;
  return mla::page_ws(nullptr, cache->num_pages, batch).total;
}

}  // extern "C"
