// mla_cache_internal.h -- parameters and launchers of the cache operators
// (include/mla_cache.h), shared by the entry points and the kernels.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "mla_cache.h"

namespace mla {

constexpr int kQueryHeads = MLA_NUM_HEADS, kLat = MLA_V_DIM, kPe = MLA_PE_DIM, kRow = MLA_QK_DIM, kPairs = MLA_PE_PAIRS;

inline int cache_row_bytes(int kv_dtype) {
  return kv_dtype == MLA_KV_BF16 ? kRow * 2 : (kv_dtype == MLA_KV_FP8_E4M3 ? kRow : kRow / 2);
}

// One layer of a cache as the row kernels see it.
struct LayerRows {
  uint8_t* kv;
  void* scale;           // fp8: fp32[1]; mxfp4: e8m0 [rows, scale_stride]
  int32_t scale_stride;
  int32_t rows;          // num_pages * page_size
};

struct AppendParams {
  LayerRows cache;
  mla_rope rope;         // num_axes 0: no rotation
  mla_norm norm;
  mla_append_args a;
  int32_t* error;
};

struct GatherParams {
  LayerRows cache;
  const int32_t* slots;
  uint8_t* out;
  int64_t out_stride;    // bytes
  int32_t num_rows;
  int32_t* error;
};

struct SlotsParams {
  mla_page_table table;
  const int32_t* qo_indptr;
  int32_t* slots;
  int32_t* rows;
  int64_t row_stride;
  int32_t num_tokens, page_shift, num_pages;
  int32_t* error;
};

// The cache as the page kernels see it.  Rows move 16 bytes at a time, scale
// rows scale_unit bytes (16, 8, 4, 2 or 1: what divides every address and length
// of the call).
struct PageBytes {
  uint8_t* kv;
  uint8_t* scale;        // mxfp4 whose scale rows fill their stride, else null
  uint8_t* scale_cols;   // mxfp4 whose scale rows are scale_width of scale_stride bytes, else null
  int64_t kv_layer, scale_layer;
  int32_t row_bytes, scale_stride, scale_width;
  int32_t page_size, page_shift, num_pages, num_layers;
  int32_t scale_unit;
};

struct CopyParams {
  PageBytes c;
  const int32_t* src;
  const int32_t* dst;
  int32_t n;
  int32_t* error;
};

// Workspace of fork / resize / compact, all int32.
struct PageWs {
  int32_t* err;          // word 0: the error word
  int32_t* head;         // kHead* words
  int32_t* first;        // [batch] first fresh place of each sequence of `to`
  int32_t* fresh;        // [batch] rank of its first fresh page
  int32_t* copy_src;     // [batch] part-filled pages to copy: the page, the rank of
  int32_t* copy_rank;    // [batch]   the fresh page that takes it,
  int32_t* copy_rows;    // [batch]   the rows in use
  int32_t* list;         // [num_pages] fresh pages by rank / pages to move into
  int32_t* from;         // [num_pages] pages to move from
  int32_t* refs;         // [num_pages] their counts
  uint32_t* mask;        // [ceil(num_pages / 32)] a bit a page: in use
  int32_t* pre;          // [ceil(num_pages / 32)] pages in use before each mask word, in its block
  int32_t* block_used;   // [ceil(num_pages / 4096)] pages in use of each block,
  int32_t* block_pre;    //   and before it
  size_t total;
};
enum { kHeadOk = 0, kHeadCopies = 1, kHeadReleases = 2, kHeadLive = 3, kHeadMoves = 4, kHeadTicket = 5 };

inline PageWs page_ws(void* base, int32_t num_pages, int32_t batch) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t pages = up(4 * (size_t)num_pages), words = up(4 * (((size_t)num_pages + 31) / 32));
  const size_t seqs = up(4 * (size_t)batch);
  uint8_t* p = static_cast<uint8_t*>(base);
  PageWs w;
  size_t at = 0;
  auto take = [&](size_t n) {
    uint8_t* q = p ? p + at : nullptr;
    at += n;
    return q;
  };
  w.err = reinterpret_cast<int32_t*>(take(256));
  w.head = reinterpret_cast<int32_t*>(take(256));
  w.first = reinterpret_cast<int32_t*>(take(seqs));
  w.fresh = reinterpret_cast<int32_t*>(take(seqs));
  w.copy_src = reinterpret_cast<int32_t*>(take(seqs));
  w.copy_rank = reinterpret_cast<int32_t*>(take(seqs));
  w.copy_rows = reinterpret_cast<int32_t*>(take(seqs));
  w.list = reinterpret_cast<int32_t*>(take(pages));
  w.from = reinterpret_cast<int32_t*>(take(pages));
  w.refs = reinterpret_cast<int32_t*>(take(pages));
  w.mask = reinterpret_cast<uint32_t*>(take(words));
  w.pre = reinterpret_cast<int32_t*>(take(words));
  const size_t blocks = up(4 * (((size_t)num_pages + 4095) / 4096));
  w.block_used = reinterpret_cast<int32_t*>(take(blocks));
  w.block_pre = reinterpret_cast<int32_t*>(take(blocks));
  w.total = at;
  return w;
}

struct TableParams {     // fork and resize
  PageBytes c;
  int32_t* refs;
  mla_page_table from, to;
  const int32_t* by;     // fork: the parent of each sequence; resize: its new length
  int32_t forks;
  int32_t entries_apart;   // the table entries are another kernel's
  PageWs ws;
};

struct CompactParams {
  PageBytes c;
  const int32_t* refs_in;
  int32_t* refs_out;
  const int32_t* idx_in;
  int32_t* idx_out;
  int32_t num_indices;
  int32_t* live;
  int32_t entries_apart;   // counts and table are another kernel's
  PageWs ws;
};

cudaError_t launch_append(const AppendParams& p, int kv_dtype, cudaStream_t s);
cudaError_t launch_gather(const GatherParams& p, int kv_dtype, cudaStream_t s);
cudaError_t launch_slots(const SlotsParams& p, cudaStream_t s);
cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t s);
cudaError_t launch_table(const TableParams& p, cudaStream_t s);
cudaError_t launch_free(int32_t* refs, int32_t num_pages, const int32_t* pages, int32_t n, int32_t* error,
                        cudaStream_t s);
cudaError_t launch_compact(const CompactParams& p, cudaStream_t s);

// Launches `kernel` so that it may begin before the stream's previous kernel has
// ended; each of these kernels waits (griddepcontrol.wait) before it reads memory.
// cluster > 0: in clusters of that many CTAs.
template <class Kernel, class Params>
inline cudaError_t launch_chained(Kernel kernel, unsigned grid, unsigned block, cudaStream_t stream, const Params& p,
                                  unsigned cluster = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace mla
