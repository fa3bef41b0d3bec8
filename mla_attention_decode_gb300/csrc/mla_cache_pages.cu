// mla_cache_pages.cu -- pages of the latent cache copied, forked, resized, freed
// and compacted (include/mla_cache.h).
//
// A call that hands out or moves pages is two kernels: one CTA decides (prefix
// sums over the sequences and over the pages' counts), then a grid carries it
// out (table entries, counts, rows).  Ranks come from prefix sums, never from
// the order in which threads arrive, so results are the same from run to run;
// the only atomics add to counts.
#include <cuda_runtime.h>

#include "mla_cache_internal.h"
#include "mla_ptx.cuh"

namespace mla {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kPlan = 1024;             // threads of a deciding CTA
constexpr unsigned kMaxGrid = 152 * 8;  // CTAs of 256 threads that carry out

__device__ __forceinline__ void set_error(int32_t* error, int32_t code) {
  if (error) *error = code;
}

// ---------------------------------------------------------------- moving rows
// A page's bytes are cut into segments of 256 units, one warp each: 8 units a
// lane, all 8 loads in flight before the first store.
constexpr int kSegUnits = 256;

__host__ __device__ inline int kv_segs(const PageBytes& c) {
  return (int)(((int64_t)c.page_size * c.row_bytes / 16 + kSegUnits - 1) / kSegUnits);
}
__host__ __device__ inline int scale_segs(const PageBytes& c) {
  return c.scale ? (int)(((int64_t)c.page_size * c.scale_stride / c.scale_unit + kSegUnits - 1) / kSegUnits) : 0;
}

template <class T>
__device__ __forceinline__ void move_units(uint8_t* dst, const uint8_t* src, int units, int lane) {
  const T* s = reinterpret_cast<const T*>(src);
  T* d = reinterpret_cast<T*>(dst);
  T v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (32 * i + lane < units) v[i] = s[32 * i + lane];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (32 * i + lane < units) d[32 * i + lane] = v[i];
}

// Segment `seg` (of kv_segs + scale_segs) of the first `rows` rows of page src
// to page dst, in layer l.
__device__ __forceinline__ void move_segment(const PageBytes& c, int src, int dst, int rows, int l, int seg, int ks,
                                             int lane) {
  if (seg < ks) {
    const int64_t page = (int64_t)c.page_size * c.row_bytes;
    const int64_t at = (int64_t)seg * (kSegUnits * 16), bytes = (int64_t)rows * c.row_bytes - at;
    if (bytes <= 0) return;
    uint8_t* base = c.kv + l * c.kv_layer + at;
    move_units<uint4>(base + dst * page, base + src * page, (int)(min(bytes, (int64_t)(kSegUnits * 16)) >> 4), lane);
    return;
  }
  const int u = c.scale_unit;
  const int64_t page = (int64_t)c.page_size * c.scale_stride;
  const int64_t at = (int64_t)(seg - ks) * kSegUnits * u, bytes = (int64_t)rows * c.scale_stride - at;
  if (bytes <= 0) return;
  const int units = (int)(min(bytes, (int64_t)kSegUnits * u) / u);
  uint8_t* base = c.scale + l * c.scale_layer + at;
  uint8_t* d = base + dst * page;
  const uint8_t* s = base + src * page;
  switch (u) {
    case 16: move_units<uint4>(d, s, units, lane); break;
    case 8: move_units<uint2>(d, s, units, lane); break;
    case 4: move_units<uint32_t>(d, s, units, lane); break;
    case 2: move_units<uint16_t>(d, s, units, lane); break;
    default: move_units<uint8_t>(d, s, units, lane); break;
  }
}

__global__ void __launch_bounds__(256) mla_copy_pages_kernel(const __grid_constant__ CopyParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int ks = kv_segs(p.c), segs = ks + scale_segs(p.c);
  const int64_t per = (int64_t)segs * p.c.num_layers, tasks = per * p.n;
  for (int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); task < tasks; task += (int64_t)gridDim.x * 8) {
    const int64_t i = task / per;
    const int rest = (int)(task - i * per), l = rest / segs, seg = rest - l * segs;
    const int src = p.src[i], dst = p.dst[i];
    if (src < 0 || src >= p.c.num_pages || dst < 0 || dst >= p.c.num_pages) {
      if (rest == 0 && lane == 0) set_error(p.error, MLA_ERR_DEVICE_INDEX);
      continue;
    }
    if (src != dst) move_segment(p.c, src, dst, p.c.page_size, l, seg, ks, lane);
  }
}

// ---------------------------------------------------------------- prefix sums
__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// Exclusive prefix sum of v over the CTA's kPlan threads, and the total.
// `part` is 33 words of shared memory; every thread of the CTA calls.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t in = warp_scan(v, lane);
  if (lane == 31) part[warp] = in;
  __syncthreads();
  if (warp == 0) {
    const int64_t x = part[lane], s = warp_scan(x, lane);
    part[lane] = s - x;
    if (lane == 31) part[32] = s;
  }
  __syncthreads();
  const int64_t ex = in - v + part[warp];
  total = part[32];
  __syncthreads();  // `part` may be written again
  return ex;
}

// The sequence that owns entry e of a table: indptr[n] <= e < indptr[n + 1].
__device__ __forceinline__ int owner(const int32_t* indptr, int batch, int e) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (indptr[mid] <= e) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------- fork, resize
// Sequence n of `to` keeps the first `first` pages of its parent and gets fresh
// pages from there on; the first of them takes a part-filled page's rows where
// that page has to be copied.
__global__ void __launch_bounds__(kPlan) mla_table_plan_kernel(const __grid_constant__ TableParams p) {
  __shared__ int64_t part[33];
  __shared__ int32_t s_bad, s_release;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int tid = threadIdx.x, N = p.to.batch, P = p.c.page_size, shift = p.c.page_shift;
  if (tid == 0) s_bad = s_release = 0;
  __syncthreads();
  int64_t pages = 0, fresh = 0, copies = 0;
  for (int base = 0; base < N; base += kPlan) {
    const int n = base + tid;
    int64_t cnt = 0;
    int32_t first = 0, src = -1, rows = 0;
    if (n < N) {
      const int par = p.forks ? p.by[n] : n;
      bool ok = par >= 0 && par < p.from.batch;
      int64_t a = 0, b = 0, len = 0, want = 0;
      if (ok) {
        a = p.from.page_indptr[par];
        b = p.from.page_indptr[par + 1];
        ok = 0 <= a && a <= b && b <= p.from.num_indices;
      }
      if (ok && b > a) {
        const int32_t last = p.from.last_page_len[par];
        ok = last >= 1 && last <= P;
        len = (b - a - 1) * P + last;
      }
      if (ok) {
        want = p.forks ? len : p.by[n];
        ok = want >= 0;
      }
      if (!ok) {
        s_bad = 1;
      } else {
        cnt = (want + P - 1) >> shift;
        const int64_t keep = min(cnt, b - a), r0 = min(len, want);
        first = (int32_t)keep;
        if ((r0 & (P - 1)) != 0 && (p.forks || want != len)) {
          const int32_t page = p.from.kv_indices[a + keep - 1];
          if (page >= 0 && page < p.c.num_pages && (p.forks || p.refs[page] > 1)) {
            src = page;
            rows = (int32_t)(r0 & (P - 1));
            first -= 1;
          }
        }
        if (!p.forks && b - a > first) s_release = 1;
        p.to.last_page_len[n] = cnt ? (int32_t)(want - (cnt - 1) * P) : 0;
        p.ws.first[n] = first;
      }
    }
    int64_t total;
    const int64_t at = block_scan(cnt, part, total);
    if (n < N) p.to.page_indptr[n + 1] = (int32_t)(pages + at + cnt);
    pages += total;
    const int64_t fr = fresh + block_scan(cnt - first, part, total);
    if (n < N) p.ws.fresh[n] = (int32_t)fr;
    fresh += total;
    const int64_t c = copies + block_scan(src >= 0, part, total);
    if (src >= 0) {
      p.ws.copy_src[c] = src;
      p.ws.copy_rank[c] = (int32_t)fr;
      p.ws.copy_rows[c] = rows;
    }
    copies += total;
  }
  int32_t err = s_bad || pages > p.to.num_indices ? MLA_ERR_DEVICE_INDEX : (fresh > p.c.num_pages ? MLA_ERR_OUT_OF_PAGES : 0);
  // the free pages of lowest number, as many as are needed
  int64_t found = 0;
  for (int base = 0; err == 0 && found < fresh && base < p.c.num_pages; base += kPlan) {
    const int pg = base + tid;
    const bool is_free = pg < p.c.num_pages && p.refs[pg] == 0;
    int64_t total;
    const int64_t k = found + block_scan(is_free, part, total);
    if (is_free && k < fresh) p.ws.list[k] = pg;
    found += total;
  }
  if (err == 0 && found < fresh) err = MLA_ERR_OUT_OF_PAGES;
  __syncthreads();
  if (err == 0) {
    for (int64_t k = tid; k < fresh; k += kPlan) p.refs[p.ws.list[k]] = 1;
    if (tid == 0) p.to.page_indptr[0] = 0;
  } else {
    for (int n = tid; n <= N; n += kPlan) {
      p.to.page_indptr[n] = 0;
      if (n < N) p.to.last_page_len[n] = 0;
    }
  }
  if (tid == 0) {
    p.ws.head[kHeadOk] = err == 0;
    p.ws.head[kHeadCopies] = (int32_t)copies;
    p.ws.head[kHeadReleases] = s_release;
    if (err) set_error(p.ws.err, err);
  }
}

__global__ void __launch_bounds__(256) mla_table_apply_kernel(const __grid_constant__ TableParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  if (!p.ws.head[kHeadOk]) return;
  const int lane = threadIdx.x & 31, N = p.to.batch;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  const int total = p.to.page_indptr[N];
  for (int64_t e = at; e < total; e += step) {
    const int n = owner(p.to.page_indptr, N, (int)e);
    const int j = (int)e - p.to.page_indptr[n], first = p.ws.first[n];
    int32_t page;
    if (j >= first) {
      page = p.ws.list[p.ws.fresh[n] + j - first];
    } else {
      page = p.from.kv_indices[p.from.page_indptr[p.forks ? p.by[n] : n] + j];
      if (page < 0 || page >= p.c.num_pages) {
        page = -1;
        set_error(p.ws.err, MLA_ERR_DEVICE_INDEX);
      } else if (p.forks) {
        atomicAdd(p.refs + page, 1);
      }
    }
    p.to.kv_indices[e] = page;
  }
  if (p.ws.head[kHeadReleases]) {  // resize: what a sequence no longer holds
    const int B = p.from.batch, end = p.from.page_indptr[B];
    for (int64_t e = p.from.page_indptr[0] + at; e < end; e += step) {
      const int n = owner(p.from.page_indptr, B, (int)e);
      if ((int)e - p.from.page_indptr[n] < p.ws.first[n]) continue;
      const int32_t page = p.from.kv_indices[e];
      if (page < 0 || page >= p.c.num_pages) {
        set_error(p.ws.err, MLA_ERR_DEVICE_INDEX);
      } else if (atomicSub(p.refs + page, 1) <= 0) {
        atomicAdd(p.refs + page, 1);
        set_error(p.ws.err, MLA_ERR_DEVICE_INDEX);
      }
    }
  }
  const int ks = kv_segs(p.c), segs = ks + scale_segs(p.c);
  const int64_t per = (int64_t)segs * p.c.num_layers, tasks = per * p.ws.head[kHeadCopies];
  for (int64_t task = at >> 5; task < tasks; task += step >> 5) {
    const int64_t i = task / per;
    const int rest = (int)(task - i * per), l = rest / segs, seg = rest - l * segs;
    move_segment(p.c, p.ws.copy_src[i], p.ws.list[p.ws.copy_rank[i]], p.ws.copy_rows[i], l, seg, ks, lane);
  }
}

// ---------------------------------------------------------------- free
struct FreeParams {
  int32_t* refs;
  const int32_t* pages;
  int32_t num_pages, n;
  int32_t* error;
};
__global__ void __launch_bounds__(256) mla_free_kernel(const __grid_constant__ FreeParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.n) return;
  const int32_t page = p.pages[i];
  if (page == -1) return;
  if (page < 0 || page >= p.num_pages) {
    set_error(p.error, MLA_ERR_DEVICE_INDEX);
  } else if (atomicSub(p.refs + page, 1) <= 0) {
    atomicAdd(p.refs + page, 1);  // given back more often than held: the count stays 0
    set_error(p.error, MLA_ERR_DEVICE_INDEX);
  }
}

// ---------------------------------------------------------------- compact
// One bit a page (in use), the pages in use before each word of 32, then the
// two lists: free pages below L, pages in use from L on.
__global__ void __launch_bounds__(kPlan) mla_compact_plan_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int64_t part[33];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pages = p.c.num_pages, words = (pages + 31) / 32;
  for (int w = warp; w < words; w += kPlan / 32) {
    const int pg = 32 * w + lane;
    const uint32_t m = __ballot_sync(kFull, pg < pages && p.refs_in[pg] > 0);
    if (lane == 0) p.ws.mask[w] = m;
  }
  __syncthreads();
  int64_t live = 0;
  for (int base = 0; base < words; base += kPlan) {
    const int w = base + tid;
    const int64_t n = w < words ? __popc(p.ws.mask[w]) : 0;
    int64_t total;
    const int64_t before = live + block_scan(n, part, total);
    if (w < words) p.ws.pre[w] = (int32_t)before;
    live += total;
  }
  __syncthreads();
  const int L = (int)live;
  // pages in use below L (L == pages: all of them)
  const int kept = L == pages ? L : p.ws.pre[L >> 5] + __popc(p.ws.mask[L >> 5] & ((1u << (L & 31)) - 1));
  for (int w = warp; w < words; w += kPlan / 32) {
    const int pg = 32 * w + lane;
    const uint32_t m = p.ws.mask[w];
    const bool used = m >> lane & 1;
    const int before = p.ws.pre[w] + __popc(m & ((1u << lane) - 1));
    if (pg < L && !used) p.ws.list[pg - before] = pg;
    if (pg >= L && used) {
      p.ws.from[before - kept] = pg;
      p.ws.refs[before - kept] = p.refs_in[pg];
    }
  }
  if (tid == 0) {
    p.ws.head[kHeadLive] = L;
    p.ws.head[kHeadMoves] = L - kept;
    if (p.live) *p.live = L;
  }
}

__global__ void __launch_bounds__(256) mla_compact_apply_kernel(const __grid_constant__ CompactParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, pages = p.c.num_pages;
  const int L = p.ws.head[kHeadLive], moves = p.ws.head[kHeadMoves], kept = L - moves;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  // pages in use before page pg, and whether pg is
  auto rank = [&](int pg, bool& used) {
    const uint32_t m = p.ws.mask[pg >> 5];
    used = m >> (pg & 31) & 1;
    return p.ws.pre[pg >> 5] + __popc(m & ((1u << (pg & 31)) - 1));
  };
  for (int64_t pg = at; pg < pages; pg += step) {
    int32_t n = 0;
    if (pg < L) {
      bool used;
      const int before = rank((int)pg, used);
      n = used ? p.refs_in[pg] : p.ws.refs[pg - before];
    }
    p.refs_out[pg] = n;
  }
  for (int64_t i = at; i < p.num_indices; i += step) {
    int32_t pg = p.idx_in[i];
    if (pg != -1) {
      bool used = false;
      const int before = pg >= 0 && pg < pages ? rank(pg, used) : 0;
      if (!used) {
        pg = -1;
        set_error(p.ws.err, MLA_ERR_DEVICE_INDEX);
      } else if (pg >= L) {
        pg = p.ws.list[before - kept];
      }
    }
    p.idx_out[i] = pg;
  }
  const int ks = kv_segs(p.c), segs = ks + scale_segs(p.c);
  const int64_t per = (int64_t)segs * p.c.num_layers, tasks = per * moves;
  for (int64_t task = at >> 5; task < tasks; task += step >> 5) {
    const int64_t i = task / per;
    const int rest = (int)(task - i * per), l = rest / segs, seg = rest - l * segs;
    move_segment(p.c, p.ws.from[i], p.ws.list[i], p.c.page_size, l, seg, ks, lane);
  }
}

// CTAs for `threads` threads of work, at most kMaxGrid (the kernels loop).
unsigned grid_for(int64_t threads) {
  const int64_t g = (threads + 255) / 256;
  return (unsigned)(g < 1 ? 1 : (g < kMaxGrid ? g : kMaxGrid));
}
int64_t copy_threads(const PageBytes& c, int64_t pages) {
  return pages * c.num_layers * (kv_segs(c) + scale_segs(c)) * 32;
}

}  // namespace

cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  return launch_chained(mla_copy_pages_kernel, grid_for(copy_threads(p.c, p.n)), 256, s, p);
}

cudaError_t launch_table(const TableParams& p, cudaStream_t s) {
  const cudaError_t e = launch_chained(mla_table_plan_kernel, 1, kPlan, s, p);
  if (e != cudaSuccess) return e;
  int64_t threads = copy_threads(p.c, p.to.batch);
  if (threads < p.to.num_indices) threads = p.to.num_indices;
  if (!p.forks && threads < p.from.num_indices) threads = p.from.num_indices;
  return launch_chained(mla_table_apply_kernel, grid_for(threads), 256, s, p);
}

cudaError_t launch_free(int32_t* refs, int32_t num_pages, const int32_t* pages, int32_t n, int32_t* error,
                        cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const FreeParams p{refs, pages, num_pages, n, error};
  return launch_chained(mla_free_kernel, (unsigned)(((int64_t)n + 255) / 256), 256, s, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t s) {
  const cudaError_t e = launch_chained(mla_compact_plan_kernel, 1, kPlan, s, p);
  if (e != cudaSuccess) return e;
  int64_t threads = copy_threads(p.c, p.c.num_pages / 2);
  if (threads < p.num_indices) threads = p.num_indices;
  if (threads < p.c.num_pages) threads = p.c.num_pages;
  return launch_chained(mla_compact_apply_kernel, grid_for(threads), 256, s, p);
}

}  // namespace mla
