// mla_cache_pages.cu -- pages of the latent cache copied, forked, resized, freed
// and compacted (include/mla_cache.h).
//
// A call that hands out or moves pages has two parts: CTAs decide (prefix sums
// over the sequences and over the pages' counts), then a grid carries it out
// (table entries, counts, rows).  Over few pages every CTA decides for itself, in
// shared memory, and carries out its share in the same launch.  Ranks come from
// prefix sums, never from the order in which threads arrive, so results are the
// same from run to run.  Atomics add to counts, gather flags, and tell which CTA
// has been the last to read counts that are rewritten in place.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "mla_cache_internal.h"
#include "mla_ptx.cuh"

namespace cg = cooperative_groups;

namespace mla {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kPlan = 512;               // threads of a deciding CTA
// Deciding CTAs.  A resize of 64 sequences of 64 pages and back takes, with the
// slots and rows between, 14.7 us with 8 CTAs, 16.3 with 4, 19.5 with 2, 25.5 with 1.
constexpr int kCluster = 8;
constexpr int kMoveCtas = 2;             // CTAs an SM that move rows (128 registers a thread)
constexpr unsigned kLocalGrid = 152 * kMoveCtas;  // all of those resident at once
constexpr unsigned kMaxGrid = 152 * 8;   // CTAs of 256 threads that carry out a call (the kernels loop)

// Which kernels a call takes; both sides of each border measured in graphs of the
// call on a GB300.
// The cluster that decides a small fork or resize also carries it out, up to this
// many table entries (8192 entries: 6.0 us against 8.3 in two launches) ...
constexpr int64_t kClusterEntries = 32768;
// ... and bytes of pages that may have to be copied: a fork of n bf16 sequences
// of 64-row pages, with its free, takes 7.4 us against 8.8 at n = 8 (0.6 MB),
// 9.5 against 9.2 at n = 16 and 32 against 12 at n = 256.  A resize copies a page
// only where a fork's sequence is cut inside a shared one.  n such cuts take 8.1 us
// against 8.5 at n = 16, 14.3 against 9.1 at n = 64 and 26.9 against 10.5 at n = 200;
// cuts that copy nothing, as most do, take 4.8 against 7.3, 5.0 against 7.8 and 5.5
// against 8.8.  The border serves those: at n = 64 one call in 3 may copy.
constexpr int64_t kClusterForkBytes = 1 << 20, kClusterResizeBytes = 16 << 20;
// Table entries by a kernel of their own: 65,536 entries 11.1 us against 10.4 in
// one with the rows, 262,144 entries 11.5 against 15.2.
constexpr int64_t kApartEntries = 131072;
// The same for a compaction's pages or entries: 200,000 pages 21.2 us against
// 20.6, 400,000 pages 32.2 against 33.5.
constexpr int64_t kApartPages = 262144;

__device__ __forceinline__ void set_error(int32_t* error, int32_t code) {
  if (error) *error = code;
}

// ---------------------------------------------------------------- moving rows
// A warp moves up to kSegUnits units of 16 bytes at a time, kDeep a lane, all
// its loads in flight before the first store.  8 a lane on 128 registers (2 CTAs
// of 256 an SM) came to 97% of the copy rate over 4001 MXFP4 pages in 6 layers
// (143 us); 4 a lane with twice the CTAs took 152 us, and 8 a lane forced into 64
// registers 182 us.
constexpr int kDeep = 8;
constexpr int kSegUnits = 32 * kDeep;

__device__ __forceinline__ uint4 load_unit(const uint8_t* p, int unit) {
  uint4 v;
  switch (unit) {
    case 16: v = *reinterpret_cast<const uint4*>(p); break;
    case 8: v.x = reinterpret_cast<const uint32_t*>(p)[0], v.y = reinterpret_cast<const uint32_t*>(p)[1]; break;
    case 4: v.x = *reinterpret_cast<const uint32_t*>(p); break;
    case 2: v.x = *reinterpret_cast<const uint16_t*>(p); break;
    default: v.x = *p; break;
  }
  return v;
}
__device__ __forceinline__ void store_unit(uint8_t* p, uint4 v, int unit) {
  switch (unit) {
    case 16: *reinterpret_cast<uint4*>(p) = v; break;
    case 8: reinterpret_cast<uint32_t*>(p)[0] = v.x, reinterpret_cast<uint32_t*>(p)[1] = v.y; break;
    case 4: *reinterpret_cast<uint32_t*>(p) = v.x; break;
    case 2: *reinterpret_cast<uint16_t*>(p) = (uint16_t)v.x; break;
    default: *p = (uint8_t)v.x; break;
  }
}

// A page's rows, then its scale rows, in segments of kSegUnits units.
__host__ __device__ inline int kv_segs(const PageBytes& c) {
  return (int)(((int64_t)c.page_size * c.row_bytes / 16 + kSegUnits - 1) / kSegUnits);
}
__host__ __device__ inline int scale_segs(const PageBytes& c) {
  return c.scale ? (int)(((int64_t)c.page_size * c.scale_stride / c.scale_unit + kSegUnits - 1) / kSegUnits) : 0;
}
// task / d and its remainder, in 32 bits where the call's tasks fit.
__device__ __forceinline__ int64_t split(int64_t task, int64_t d, bool narrow, int64_t& rest) {
  const int64_t q = narrow ? (int64_t)((uint32_t)task / (uint32_t)d) : task / d;
  rest = task - q * d;
  return q;
}

// The first rows of part-filled pages: part(i) -> (source, destination, rows),
// i < n, in every layer.  Forks of one sequence follow one another and copy the
// same page: a warp takes up to kShare copies in a row, as far as there are
// warps' worth of them, and reads a source once.  A fork of 64 sequences into 512
// that copies 102 MB in 12 layers, with its free: 45.0 us with one copy a warp,
// 38.5 with 2, 35.8 with 4 and 35.6 with 8; 33.1 with 4 and 3 CTAs an SM instead of
// 2 (4 CTAs: 35.1).
constexpr int kShare = 4;
constexpr int kPartCtas = 3;  // CTAs an SM of the kernel that does this
template <class Part>
__device__ __forceinline__ void move_parts(const PageBytes& c, int n, int64_t at, int64_t step, Part part) {
  const int lane = threadIdx.x & 31, ks = kv_segs(c), segs = ks + scale_segs(c);
  const int64_t per = (int64_t)segs * c.num_layers, warps = step >> 5;
  const int share = (int)max((int64_t)1, min((int64_t)kShare, per * n / warps));
  const int64_t tasks = per * ((n + share - 1) / share);
  const bool narrow = tasks <= UINT32_MAX;
  for (int64_t task = at >> 5; task < tasks; task += warps) {
    int64_t rest, seg;
    const int i0 = (int)split(task, per, narrow, rest) * share, many = min(share, n - i0);
    const int64_t l = split(rest, segs, true, seg);
    const int3 mine = part(i0 + min(lane, many - 1));  // all the copies' pages in one round
    const bool kv = seg < ks;
    const int unit = kv ? 16 : c.scale_unit;
    const int64_t row = kv ? c.row_bytes : c.scale_stride, page = c.page_size * row;
    const int64_t off = (kv ? seg : seg - ks) * kSegUnits * unit;
    uint8_t* base = (kv ? c.kv + l * c.kv_layer : c.scale + l * c.scale_layer) + off + (int64_t)lane * unit;
    uint4 v[kDeep];
    int src = -1, rows = -1, units = 0;
    for (int i = 0; i < many; ++i) {
      const int from = __shfl_sync(kFull, mine.x, i), to = __shfl_sync(kFull, mine.y, i);
      const int used = __shfl_sync(kFull, mine.z, i);
      if (from != src || used != rows) {
        const int64_t bytes = used * row - off;
        units = bytes <= 0 ? 0 : (int)(min(bytes, (int64_t)kSegUnits * unit) / unit);
        const uint8_t* s = base + from * page;
        if (unit == 16) {
#pragma unroll
          for (int k = 0; k < kDeep; ++k)
            if (32 * k + lane < units) v[k] = reinterpret_cast<const uint4*>(s)[32 * k];
        } else {
#pragma unroll
          for (int k = 0; k < kDeep; ++k)
            if (32 * k + lane < units) v[k] = load_unit(s + 32 * k * unit, unit);
        }
        src = from;
        rows = used;
      }
      uint8_t* d = base + to * page;
      if (unit == 16) {
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
          if (32 * k + lane < units) reinterpret_cast<uint4*>(d)[32 * k] = v[k];
      } else {
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
          if (32 * k + lane < units) store_unit(d + 32 * k * unit, v[k], unit);
      }
    }
  }
}

// Whole pages: page pair(i) -> (src, dst), i < n, in every layer (src < 0: none).
// A page and its scale rows are one run of 16-byte units where the latter divide
// into them; a page of up to kSegUnits units is moved by 4 to 32 lanes, so that
// a warp has several small pages in flight (a page of one MXFP4 row is 18 units
// and nine of 2 bytes).  `at`: the thread's index of `step`, both over warps.
template <class Pair>
__device__ __forceinline__ void move_pages(const PageBytes& c, int64_t n, int64_t at, int64_t step, Pair pair) {
  const int lane = threadIdx.x & 31, unit = c.scale_unit;
  const int64_t kv_page = (int64_t)c.page_size * c.row_bytes;
  const int64_t scale_page = c.scale ? (int64_t)c.page_size * c.scale_stride : 0;
  const int64_t kvu = kv_page / 16, su = unit == 16 ? 0 : scale_page / unit;
  const int64_t units = kvu + (unit == 16 ? scale_page / 16 : 0);
  const int64_t warp = at >> 5, warps = step >> 5;
  if (units <= kSegUnits) {
    int g = 4;  // lanes a page
    while (g * kDeep < units) g *= 2;
    const int sub = lane / g, gl = lane - sub * g;
    const int64_t tasks = n * c.num_layers;
    const bool narrow = tasks <= UINT32_MAX;
    for (int64_t task = warp * (32 / g) + sub; task < tasks; task += warps * (32 / g)) {
      int64_t l;
      const int64_t i = split(task, c.num_layers, narrow, l);
      const int2 p = pair(i, l == 0 && gl == 0);
      if (p.x < 0) continue;
      uint8_t* kv = c.kv + l * c.kv_layer;
      uint8_t* sc = c.scale + l * c.scale_layer;
      uint4 v[kDeep], w[3];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int64_t u = k * g + gl;
        if (u < units)
          v[k] = *reinterpret_cast<const uint4*>(u < kvu ? kv + p.x * kv_page + 16 * u
                                                         : sc + p.x * scale_page + 16 * (u - kvu));
      }
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k * g + gl < su) w[k] = load_unit(sc + p.x * scale_page + (k * g + gl) * unit, unit);
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int64_t u = k * g + gl;
        if (u < units)
          *reinterpret_cast<uint4*>(u < kvu ? kv + p.y * kv_page + 16 * u
                                            : sc + p.y * scale_page + 16 * (u - kvu)) = v[k];
      }
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k * g + gl < su) store_unit(sc + p.y * scale_page + (k * g + gl) * unit, w[k], unit);
      for (int64_t u = 3 * g + gl; u < su; u += g)  // (scale rows of odd strides)
        store_unit(sc + p.y * scale_page + u * unit, load_unit(sc + p.x * scale_page + u * unit, unit), unit);
    }
    return;
  }
  const int64_t us = (units + kSegUnits - 1) / kSegUnits, segs = us + (su + kSegUnits - 1) / kSegUnits;
  const int64_t per = segs * c.num_layers, tasks = per * n;
  const bool narrow = tasks <= UINT32_MAX;
  for (int64_t task = warp; task < tasks; task += warps) {
    int64_t rest, seg;
    const int64_t i = split(task, per, narrow, rest), l = split(rest, segs, narrow, seg);
    const int2 p = pair(i, rest == 0 && lane == 0);
    if (p.x < 0) continue;
    uint8_t* kv = c.kv + l * c.kv_layer;
    uint8_t* sc = c.scale + l * c.scale_layer;
    uint4 v[kDeep];
    if (seg < us) {
      const int64_t u0 = seg * kSegUnits + lane;
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int64_t u = u0 + 32 * k;
        if (u < units)
          v[k] = *reinterpret_cast<const uint4*>(u < kvu ? kv + p.x * kv_page + 16 * u
                                                         : sc + p.x * scale_page + 16 * (u - kvu));
      }
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int64_t u = u0 + 32 * k;
        if (u < units)
          *reinterpret_cast<uint4*>(u < kvu ? kv + p.y * kv_page + 16 * u
                                            : sc + p.y * scale_page + 16 * (u - kvu)) = v[k];
      }
    } else {
      const int64_t u0 = (seg - us) * kSegUnits + lane;
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
        if (u0 + 32 * k < su) v[k] = load_unit(sc + p.x * scale_page + (u0 + 32 * k) * unit, unit);
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
        if (u0 + 32 * k < su) store_unit(sc + p.y * scale_page + (u0 + 32 * k) * unit, v[k], unit);
    }
  }
}

__global__ void __launch_bounds__(256, kMoveCtas) mla_copy_pages_kernel(const __grid_constant__ CopyParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  move_pages(p.c, p.n, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256, [&](int64_t i, bool tell) {
    const int src = p.src[i], dst = p.dst[i];
    const bool ok = src >= 0 && src < p.c.num_pages && dst >= 0 && dst < p.c.num_pages;
    if (!ok && tell) set_error(p.error, MLA_ERR_DEVICE_INDEX);
    return ok && src != dst ? make_int2(src, dst) : make_int2(-1, -1);
  });
}

// Scale rows that are some columns of a wider tensor: only those columns are the
// cache's, so the rows do not move in runs with what lies between them.  A thread
// a row: move(i) -> (source, destination, rows), i < n, in every layer.  This is a
// launch of its own after the one that moves the keys' rows.
template <class Move>
__device__ __forceinline__ void move_scale_columns(const PageBytes& c, int64_t n, Move move) {
  const int64_t step = (int64_t)gridDim.x * 256, per = (int64_t)c.page_size * c.num_layers;
  for (int64_t task = (int64_t)blockIdx.x * 256 + threadIdx.x; task < n * per; task += step) {
    const int64_t i = task / per, rest = task - i * per, l = rest >> c.page_shift, row = rest & (c.page_size - 1);
    const int3 m = move(i);
    if (m.x < 0 || row >= m.z) continue;
    uint8_t* base = c.scale_cols + l * c.scale_layer;
    const uint8_t* src = base + ((int64_t)m.x * c.page_size + row) * c.scale_stride;
    uint8_t* dst = base + ((int64_t)m.y * c.page_size + row) * c.scale_stride;
    for (int at = 0; at < c.scale_width; at += c.scale_unit)
      store_unit(dst + at, load_unit(src + at, c.scale_unit), c.scale_unit);
  }
}
__global__ void __launch_bounds__(256) mla_copy_scale_columns_kernel(const __grid_constant__ CopyParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  move_scale_columns(p.c, p.n, [&](int64_t i) {
    const int src = p.src[i], dst = p.dst[i];
    const bool ok = src >= 0 && src < p.c.num_pages && dst >= 0 && dst < p.c.num_pages && src != dst;
    return make_int3(ok ? src : -1, dst, p.c.page_size);
  });
}
__global__ void __launch_bounds__(256) mla_table_scale_columns_kernel(const __grid_constant__ TableParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  if (!p.ws.head[kHeadOk]) return;
  move_scale_columns(p.c, p.ws.head[kHeadCopies], [&](int64_t i) {
    return make_int3(p.ws.copy_src[i], p.ws.list[p.ws.copy_rank[i]], p.ws.copy_rows[i]);
  });
}
__global__ void __launch_bounds__(256) mla_compact_scale_columns_kernel(const __grid_constant__ CompactParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  move_scale_columns(p.c, p.ws.head[kHeadMoves],
                     [&](int64_t i) { return make_int3(p.ws.from[i], p.ws.list[i], p.c.page_size); });
}

// ---------------------------------------------------------------- prefix sums
// Exclusive prefix sums of kN values over the CTA's kThreads threads, and the
// totals.  Every thread of the CTA calls.
template <int kN, class T, int kThreads = kPlan>
struct Scan {
  static constexpr int kWarps = kThreads / 32;
  T part[kN][kWarps], total[kN];
  __device__ __forceinline__ void run(T (&v)[kN], T (&sum)[kN]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T in[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) in[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const T u = __shfl_up_sync(kFull, in[k], o);
        if (lane >= o) in[k] += u;
      }
    if (lane == 31)
#pragma unroll
      for (int k = 0; k < kN; ++k) part[k][warp] = in[k];
    __syncthreads();
    if (warp < kN) {  // warp k scans value k's warp totals
      const T x = lane < kWarps ? part[warp][lane] : T(0);
      T s = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(kFull, s, o);
        if (lane >= o) s += u;
      }
      if (lane < kWarps) part[warp][lane] = s - x;
      if (lane == 31) total[warp] = s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      v[k] = in[k] - v[k] + part[k][warp];
      sum[k] = total[k];
    }
    __syncthreads();  // the arrays may be written again
  }
};

// A page that a table may name: in range, and held (`used`: a bit a page).
__device__ __forceinline__ bool is_held(const uint32_t* used, int num_pages, int32_t page) {
  return page >= 0 && page < num_pages && (used[page >> 5] >> (page & 31) & 1);
}
// One hold on a page ends.  A page given back more often than it is held keeps
// the count 0.
__device__ __forceinline__ void release_page(int32_t* refs, int num_pages, int32_t page, int32_t* error) {
  if (page < 0 || page >= num_pages) {
    set_error(error, MLA_ERR_DEVICE_INDEX);
  } else if (atomicSub(refs + page, 1) <= 0) {
    atomicAdd(refs + page, 1);
    set_error(error, MLA_ERR_DEVICE_INDEX);
  }
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

// ---------------------------------------------------------------- pages in use
// Four counts from page pg on, `other` past the end.
__device__ __forceinline__ int4 four_counts(const int32_t* refs, int pg, int pages, int other) {
  if (pg + 4 <= pages) return *reinterpret_cast<const int4*>(refs + pg);
  int4 v = make_int4(other, other, other, other);
  if (pg < pages) v.x = refs[pg];
  if (pg + 1 < pages) v.y = refs[pg + 1];
  if (pg + 2 < pages) v.z = refs[pg + 2];
  return v;
}
// Two lanes' four bits each to a byte of the mask.
__device__ __forceinline__ void put_nibble(uint8_t* bytes, int quad, uint32_t nib) {
  const uint32_t next = __shfl_down_sync(kFull, nib, 1);
  if ((quad & 1) == 0) bytes[quad / 2] = (uint8_t)(nib | next << 4);
}

// One bit a page (its count is above 0) in mask[], in blocks of kBlock pages, 8 a
// thread: the bits before word w in its block are in pre[w], the block's in
// block_used[b].  The rank of a free page follows too: free pages before page x
// = x - pages in use before x.
constexpr int kBlock = 8 * kPlan;  // pages
struct Blocks {
  Scan<1, int32_t> scan;
  int32_t before[kPlan];  // pages in use before each of kPlan blocks,
  int32_t used[kPlan];    //   and in it
};
__device__ __forceinline__ void mask_block(const PageWs& ws, const int32_t* refs, int pages, int b, Blocks& s) {
  const int tid = threadIdx.x, base = b * kBlock, here = min(kBlock, pages - base);
  const int4 x = four_counts(refs + base, 8 * tid, here, 0), y = four_counts(refs + base, 8 * tid + 4, here, 0);
  const uint32_t m = (uint32_t)(x.x > 0) | (uint32_t)(x.y > 0) << 1 | (uint32_t)(x.z > 0) << 2 |
                     (uint32_t)(x.w > 0) << 3 | (uint32_t)(y.x > 0) << 4 | (uint32_t)(y.y > 0) << 5 |
                     (uint32_t)(y.z > 0) << 6 | (uint32_t)(y.w > 0) << 7;
  int32_t v[1] = {__popc(m)}, sum[1];
  s.scan.run(v, sum);
  const int i = b * kPlan + tid;
  if ((8 * tid & ~31) < here) {  // whole words, so that their last bits are 0
    reinterpret_cast<uint8_t*>(ws.mask)[i] = (uint8_t)m;
    if ((tid & 3) == 0) ws.pre[i >> 2] = v[0];
  }
  if (tid == 0) ws.block_used[b] = sum[0];
}
// This thread's 8 pages of block b: the first, their bits, the pages in use before it.
struct Eight {
  int64_t page;
  uint32_t used;
  int32_t before;
  __device__ __forceinline__ Eight(const PageWs& ws, int b, int32_t before_block, int64_t pages) {
    const int i = b * kPlan + threadIdx.x, shift = (i & 3) * 8;
    page = 8ll * i;
    used = 0;
    before = 0;
    if (page >= pages) return;
    const uint32_t word = ws.mask[i >> 2];
    used = word >> shift & 255u;
    before = before_block + ws.pre[i >> 2] + __popc(word & ((1u << shift) - 1));
  }
};
__host__ __device__ inline int blocks_of(int32_t pages) { return (int)(((int64_t)pages + kBlock - 1) / kBlock); }

// A CTA per block, for caches of more blocks than the deciding cluster has CTAs
// (1,049,444 pages: the cluster alone read their counts in 25 us).
struct MaskParams {
  PageWs ws;
  const int32_t* refs;
  int32_t pages;
};
__global__ void __launch_bounds__(kPlan) mla_mask_kernel(const __grid_constant__ MaskParams p) {
  __shared__ Blocks s;
  pdl_wait_primary();
  pdl_launch_dependents();
  mask_block(p.ws, p.refs, p.pages, blockIdx.x, s);
}

// ---------------------------------------------------------------- fork, resize
// Sequence n of `to` keeps the first `first` pages of its parent and gets fresh
// pages from there on; the first of them takes a part-filled page's rows where
// that page has to be copied.

// What a call does with sequence n.
struct SeqPlan {
  int64_t a, b;       // its parent's entries in `from`
  int64_t cnt;        // its pages
  int64_t want;       // its rows
  int32_t first;      // the first fresh one
  int32_t src, rows;  // the part-filled page whose rows that one takes (-1: none)
  bool ok, release;   // the parent's pages from `first` on are given back
};
__device__ __forceinline__ SeqPlan plan_sequence(const TableParams& p, int n) {
  const int P = p.c.page_size;
  SeqPlan s;
  s.a = s.b = s.cnt = s.want = 0;
  s.first = s.rows = 0;
  s.src = -1;
  s.release = false;
  const int by = p.by[n], par = p.forks ? by : n;
  s.ok = par >= 0 && par < p.from.batch;
  if (!s.ok) return s;
  s.a = p.from.page_indptr[par];
  s.b = p.from.page_indptr[par + 1];
  const int32_t last = p.from.last_page_len[par];
  const int64_t len = s.a < s.b ? (s.b - s.a - 1) * P + last : 0;
  s.want = p.forks ? len : by;
  s.ok = 0 <= s.a && s.a <= s.b && s.b <= p.from.num_indices && (s.a == s.b || (last >= 1 && last <= P)) && s.want >= 0;
  if (!s.ok) return s;
  s.cnt = (s.want + P - 1) >> p.c.page_shift;
  const int64_t keep = min(s.cnt, s.b - s.a), r0 = min(len, s.want);
  s.first = (int32_t)keep;
  if ((r0 & (P - 1)) != 0 && (p.forks || s.want != len)) {
    const int32_t page = p.from.kv_indices[s.a + keep - 1];
    if (page >= 0 && page < p.c.num_pages && p.refs[page] > (p.forks ? 0 : 1)) {
      s.src = page;
      s.rows = (int32_t)(r0 & (P - 1));
      s.first -= 1;
    }
  }
  s.release = !p.forks && s.b - s.a > s.first;
  return s;
}
// The rows in the last of cnt pages that hold `want` rows.
__device__ __forceinline__ int32_t last_rows(int64_t want, int64_t cnt, int P) {
  return cnt ? (int32_t)(want - (cnt - 1) * P) : 0;
}

// What the first CTA of the cluster decides.
struct TableTotals {
  int64_t pages, fresh, copies;
  int32_t bad, release;
};
__device__ __forceinline__ void plan_sequences(const TableParams& p, Scan<3, int64_t>& scan, TableTotals& s) {
  const int tid = threadIdx.x, N = p.to.batch;
  if (tid == 0) s.bad = s.release = 0;
  __syncthreads();
  int64_t pages = 0, fresh = 0, copies = 0;
  for (int base = 0; base < N; base += kPlan) {
    const int n = base + tid;
    SeqPlan q;
    q.cnt = q.first = 0;
    q.src = -1;
    if (n < N) {
      q = plan_sequence(p, n);
      if (!q.ok) s.bad = 1;
      if (q.release) s.release = 1;
      p.to.last_page_len[n] = last_rows(q.want, q.cnt, p.c.page_size);
      p.ws.first[n] = q.first;
    }
    int64_t v[3] = {q.cnt, q.cnt - q.first, q.src >= 0}, sum[3];
    scan.run(v, sum);
    const int64_t fr = fresh + v[1], c = copies + v[2];
    if (n < N) {
      p.to.page_indptr[n + 1] = (int32_t)(pages + v[0] + q.cnt);
      p.ws.fresh[n] = (int32_t)fr;
    }
    if (q.src >= 0) {
      p.ws.copy_src[c] = q.src;
      p.ws.copy_rank[c] = (int32_t)fr;
      p.ws.copy_rows[c] = q.rows;
    }
    pages += sum[0];
    fresh += sum[1];
    copies += sum[2];
  }
  if (tid == 0) {
    p.to.page_indptr[0] = 0;
    s.pages = pages;
    s.fresh = fresh;
    s.copies = copies;
  }
}

// Carries a decided call out: table entries and the counts of shared pages, and
// what a resized sequence no longer holds ...
__device__ __forceinline__ void apply_entries(const TableParams& p, int64_t at, int64_t step) {
  const int N = p.to.batch;
  const int total = p.to.page_indptr[N];
  for (int64_t e = at; e < total; e += step) {
    const int n = owner(p.to.page_indptr, N, (int)e);
    const int j = (int)e - p.to.page_indptr[n], first = p.ws.first[n];
    int32_t page;
    if (j >= first) {
      page = p.ws.list[p.ws.fresh[n] + j - first];
    } else {
      page = p.from.kv_indices[p.from.page_indptr[p.forks ? p.by[n] : n] + j];
      if (!is_held(p.ws.mask, p.c.num_pages, page)) {
        page = -1;
        set_error(p.ws.err, MLA_ERR_DEVICE_INDEX);
      } else if (p.forks) {
        atomicAdd(p.refs + page, 1);
      }
    }
    p.to.kv_indices[e] = page;
  }
  if (p.ws.head[kHeadReleases]) {
    const int B = p.from.batch, end = p.from.page_indptr[B];
    for (int64_t e = p.from.page_indptr[0] + at; e < end; e += step) {
      const int n = owner(p.from.page_indptr, B, (int)e);
      if ((int)e - p.from.page_indptr[n] < p.ws.first[n]) continue;
      const int32_t page = p.from.kv_indices[e];
      if (is_held(p.ws.mask, p.c.num_pages, page)) release_page(p.refs, p.c.num_pages, page, p.ws.err);
      else set_error(p.ws.err, MLA_ERR_DEVICE_INDEX);
    }
  }
}
// ... and the rows of part-filled pages.
__device__ __forceinline__ void apply_copies(const TableParams& p, int64_t at, int64_t step) {
  move_parts(p.c, p.ws.head[kHeadCopies], at, step, [&](int i) {
    return make_int3(p.ws.copy_src[i], p.ws.list[p.ws.copy_rank[i]], p.ws.copy_rows[i]);
  });
}

// The first CTA goes over the sequences, all of them over the pages (where
// mla_mask_kernel has not), and then list the free pages of lowest number, as
// many as are needed.
__global__ void __launch_bounds__(kPlan, 1) mla_table_plan_kernel(const __grid_constant__ TableParams p) {
  __shared__ Scan<3, int64_t> scan;
  __shared__ Blocks s;
  __shared__ TableTotals s_tot;
  pdl_wait_primary();
  pdl_launch_dependents();
  const cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int pages = p.c.num_pages, blocks = blocks_of(pages);
  if (blocks <= kCluster)
    for (int b = ctas - 1 - rank; b < blocks; b += ctas) mask_block(p.ws, p.refs, pages, b, s);
  if (rank == 0) plan_sequences(p, scan, s_tot);
  cluster.sync();
  const TableTotals tot = *cluster.map_shared_rank(&s_tot, 0);
  int32_t used = 0;  // before the blocks of this pass
  int32_t err = tot.bad || tot.pages > p.to.num_indices ? MLA_ERR_DEVICE_INDEX : 0;
  // every page in use, by all threads of each CTA
  int32_t all[1] = {0}, sum[1];
  for (int b = tid; b < blocks; b += kPlan) all[0] += p.ws.block_used[b];
  s.scan.run(all, sum);
  if (err == 0 && tot.fresh > pages - sum[0]) err = MLA_ERR_OUT_OF_PAGES;
  if (err == 0) {
    for (int base = 0; base < blocks; base += kPlan) {
      int32_t v[1] = {base + tid < blocks ? p.ws.block_used[base + tid] : 0};
      s.used[tid] = v[0];
      s.scan.run(v, sum);
      s.before[tid] = used + v[0];
      __syncthreads();
      const int last = min(blocks - base, kPlan);
      for (int i = rank; i < last; i += ctas) {
        const int b = base + i;
        if ((int64_t)b * kBlock - s.before[i] >= tot.fresh) break;  // so are the blocks after it
        if (s.used[i] == kBlock) continue;                          // no free page
        const Eight e(p.ws, b, s.before[i], pages);
        if (e.page >= pages) continue;
        uint32_t m = ~e.used & 255u;
        if (pages - e.page < 8) m &= (1u << (pages - e.page)) - 1;
        for (int64_t k = e.page - e.before; m != 0 && k < tot.fresh; ++k) {
          const int32_t free_page = (int32_t)e.page + __ffs(m) - 1;
          m &= m - 1;
          p.ws.list[k] = free_page;
          p.refs[free_page] = 1;
        }
      }
      used += sum[0];
      __syncthreads();
    }
  }
  if (rank == 0) {
    if (err) {
      for (int n = tid; n <= p.to.batch; n += kPlan) {
        p.to.page_indptr[n] = 0;
        if (n < p.to.batch) p.to.last_page_len[n] = 0;
      }
      if (tid == 0) set_error(p.ws.err, err);
    }
    if (tid == 0) {
      p.ws.head[kHeadOk] = err == 0;
      p.ws.head[kHeadCopies] = (int32_t)tot.copies;
      p.ws.head[kHeadReleases] = tot.release;
    }
  }
  cluster.sync();  // the first CTA's shared memory stays until the others have read it
}

__global__ void __launch_bounds__(256, kPartCtas) mla_table_apply_kernel(const __grid_constant__ TableParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  if (!p.ws.head[kHeadOk]) return;
  // every fourth CTA (the grid is a multiple of 4) has entries, a chain of
  // dependent reads each, while the others keep the rows moving
  const int64_t quarter = blockIdx.x >> 2, entry_ctas = p.entries_apart ? 0 : gridDim.x >> 2;
  if (entry_ctas > 0 && (blockIdx.x & 3) == 0)
    apply_entries(p, quarter * 256 + threadIdx.x, entry_ctas * 256);
  else
    apply_copies(p, (blockIdx.x - (entry_ctas > 0 ? quarter + 1 : 0)) * 256 + threadIdx.x,
                 (gridDim.x - entry_ctas) * 256);
}
// Long tables apart from the rows: moving rows takes 80 registers a thread and 3
// CTAs an SM, under half of the threads that a chain of dependent reads per entry
// wants (32 registers here, 8 CTAs an SM).
__global__ void __launch_bounds__(256) mla_table_entries_kernel(const __grid_constant__ TableParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  if (p.ws.head[kHeadOk]) apply_entries(p, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// Small calls (up to kPlan sequences, kLocalPages pages): each CTA of the cluster
// decides the whole call for itself, in shared memory, and carries out its
// share; nothing is handed from CTA to CTA and nothing else is launched.  Only
// the counts may not change before every CTA has read them: the cluster's barrier.
constexpr int kLocalPages = 16384;  // 32 a thread
struct TableLocal {
  Scan<4, int32_t> scan;
  int32_t to_at[kPlan + 1], from_at[kPlan + 1], first[kPlan], fresh[kPlan];
  int32_t copy_rows[kPlan];
  uint16_t copy_src[kPlan], copy_rank[kPlan];
  int32_t flags;
  union {
    uint8_t bytes[kLocalPages / 8];  // a bit a page: in use
    uint32_t words[kLocalPages / 32];
  } mask;
  uint16_t list[kLocalPages];
};
static_assert(sizeof(TableLocal) <= 48 * 1024, "static shared memory");

__global__ void __launch_bounds__(kPlan, 1) mla_table_local_kernel(const __grid_constant__ TableParams p) {
  __shared__ TableLocal s;
  pdl_wait_primary();
  pdl_launch_dependents();
  const cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)cluster.block_rank(), N = p.to.batch;
  const int pages = p.c.num_pages;
  constexpr int kPasses = kLocalPages / (4 * kPlan);
  if (tid == 0) s.flags = 0;
  int4 c4[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) c4[i] = four_counts(p.refs, (i * kPlan + tid) * 4, pages, 1);
  SeqPlan q;
  q.cnt = q.first = 0;
  q.src = -1;
  q.ok = true;
  q.release = false;
  if (tid < N) q = plan_sequence(p, tid);
  // more pages than `to` has room for: the sums below fit 32 bits without it
  if (q.cnt > p.to.num_indices) q.ok = false;
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    put_nibble(s.mask.bytes, i * kPlan + tid,
               (uint32_t)(c4[i].x > 0) | (uint32_t)(c4[i].y > 0) << 1 | (uint32_t)(c4[i].z > 0) << 2 |
                   (uint32_t)(c4[i].w > 0) << 3);
  __syncthreads();
  if (!q.ok) atomicOr(&s.flags, 1);
  if (q.release) atomicOr(&s.flags, 2);
  uint32_t m = ~s.mask.words[tid];  // the free pages
  int32_t v[4] = {q.ok ? (int32_t)q.cnt : 0, q.ok ? (int32_t)(q.cnt - q.first) : 0, q.ok && q.src >= 0, __popc(m)};
  int32_t sum[4];
  s.scan.run(v, sum);
  const int32_t total = sum[0], fresh = sum[1], copies = sum[2];
  const bool bad = (s.flags & 1) != 0 || total > p.to.num_indices;
  const int32_t err = bad ? MLA_ERR_DEVICE_INDEX : (fresh > sum[3] ? MLA_ERR_OUT_OF_PAGES : 0);
  if (tid < N) {
    s.to_at[tid] = v[0];
    s.from_at[tid] = (int32_t)q.a;
    s.first[tid] = q.first;
    s.fresh[tid] = v[1];
    if (tid == N - 1) {
      s.to_at[N] = total;
      s.from_at[N] = (int32_t)q.b;
    }
    if (q.src >= 0) {
      s.copy_src[v[2]] = (uint16_t)q.src;
      s.copy_rank[v[2]] = (uint16_t)v[1];
      s.copy_rows[v[2]] = q.rows;
    }
    if (rank == 0) {
      p.to.page_indptr[tid] = err ? 0 : v[0];
      p.to.last_page_len[tid] = err ? 0 : last_rows(q.want, q.cnt, p.c.page_size);
    }
  }
  if (rank == 0 && tid == 0) {
    p.to.page_indptr[N] = err ? 0 : total;
    if (err) set_error(p.ws.err, err);
  }
  for (int32_t k = v[3]; m != 0 && k < fresh; ++k) {
    s.list[k] = (uint16_t)(32 * tid + __ffs(m) - 1);
    m &= m - 1;
  }
  cluster.sync();  // this CTA's shared memory is written, every CTA has read the counts
  if (err) return;
  const int at = rank * kPlan + tid, step = (int)cluster.num_blocks() * kPlan;
  for (int e = at; e < total; e += step) {
    const int n = owner(s.to_at, N, e), j = e - s.to_at[n], first = s.first[n];
    int32_t page;
    if (j >= first) {
      page = s.list[s.fresh[n] + j - first];
    } else {
      page = p.from.kv_indices[s.from_at[n] + j];
      if (!is_held(s.mask.words, pages, page)) {
        page = -1;
        set_error(p.ws.err, MLA_ERR_DEVICE_INDEX);
      } else if (p.forks) {
        atomicAdd(p.refs + page, 1);
      }
    }
    p.to.kv_indices[e] = page;
  }
  for (int k = at; k < fresh; k += step) p.refs[s.list[k]] = 1;
  if (s.flags & 2)
    for (int e = s.from_at[0] + at; e < s.from_at[N]; e += step) {
      const int n = owner(s.from_at, N, e);
      if (e - s.from_at[n] < s.first[n]) continue;
      const int32_t page = p.from.kv_indices[e];
      if (is_held(s.mask.words, pages, page)) release_page(p.refs, pages, page, p.ws.err);
      else set_error(p.ws.err, MLA_ERR_DEVICE_INDEX);
    }
  move_parts(p.c, copies, at, step,
             [&](int i) { return make_int3(s.copy_src[i], s.list[s.copy_rank[i]], s.copy_rows[i]); });
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
  if (page != -1) release_page(p.refs, p.num_pages, page, p.error);
}

// ---------------------------------------------------------------- compact
// The pages in use before each block, then the two lists: free pages below L,
// pages in use from L on.  Every CTA sums the blocks for itself, so where
// mla_mask_kernel has gone over the pages any number of CTAs can share the lists.
__global__ void __launch_bounds__(kPlan, 1) mla_compact_plan_kernel(const __grid_constant__ CompactParams p) {
  __shared__ Blocks s;
  pdl_wait_primary();
  pdl_launch_dependents();
  const cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)blockIdx.x, ctas = (int)gridDim.x;
  const int pages = p.c.num_pages, blocks = blocks_of(pages);
  if (blocks <= kCluster) {  // the grid is one cluster
    for (int b = rank; b < blocks; b += ctas) mask_block(p.ws, p.refs_in, pages, b, s);
    cluster.sync();
  }
  int32_t v[1] = {0}, sum[1];
  for (int b = tid; b < blocks; b += kPlan) v[0] += p.ws.block_used[b];
  s.scan.run(v, sum);
  const int L = sum[0];
  int kept = L;  // pages in use below L (L == pages: all of them)
  if (L < pages) {
    v[0] = 0;
    for (int b = tid; b < L / kBlock; b += kPlan) v[0] += p.ws.block_used[b];
    s.scan.run(v, sum);
    kept = sum[0] + p.ws.pre[L >> 5] + __popc(p.ws.mask[L >> 5] & ((1u << (L & 31)) - 1));
  }
  int32_t used = 0;
  for (int base = 0; base < blocks; base += kPlan) {
    v[0] = base + tid < blocks ? p.ws.block_used[base + tid] : 0;
    s.used[tid] = v[0];
    s.scan.run(v, sum);
    s.before[tid] = used + v[0];
    if (rank == 0 && base + tid < blocks) p.ws.block_pre[base + tid] = used + v[0];
    __syncthreads();
    const int last = min(blocks - base, kPlan);
    for (int i = rank; i < last; i += ctas) {
      // nothing to list: full and below L, or empty and from L on
      const int64_t first = (int64_t)(base + i) * kBlock;
      if (s.used[i] == (first + kBlock <= L ? kBlock : (first >= L ? 0 : -1))) continue;
      const Eight e(p.ws, base + i, s.before[i], pages);
      // below L the free pages, from L on those in use
      const uint32_t below = e.page + 8 <= L ? 255u : (e.page >= L ? 0u : (1u << (L - e.page)) - 1);
      for (uint32_t f = ~e.used & below; f != 0; f &= f - 1) {
        const int j = __ffs(f) - 1;
        p.ws.list[(int32_t)e.page + j - (e.before + __popc(e.used & ((1u << j) - 1)))] = (int32_t)e.page + j;
      }
      int at = e.before + __popc(e.used & below) - kept;
      for (uint32_t f = e.used & ~below; f != 0; f &= f - 1, ++at) {
        const int32_t page = (int32_t)e.page + __ffs(f) - 1;
        p.ws.from[at] = page;
        p.ws.refs[at] = p.refs_in[page];
      }
    }
    used += sum[0];
    __syncthreads();
  }
  if (rank == 0 && tid == 0) {
    p.ws.head[kHeadLive] = L;
    p.ws.head[kHeadMoves] = L - kept;
    if (p.live) *p.live = L;
  }
}

// The counts and the table by the pages' new numbers ...
__device__ __forceinline__ void compact_entries(const CompactParams& p, int64_t at, int64_t step) {
  const int pages = p.c.num_pages;
  const int L = p.ws.head[kHeadLive], kept = L - p.ws.head[kHeadMoves];
  // pages in use before page pg, and whether pg is
  auto rank = [&](int pg, bool& used) {
    const uint32_t m = p.ws.mask[pg >> 5];
    used = m >> (pg & 31) & 1;
    return p.ws.block_pre[pg / kBlock] + p.ws.pre[pg >> 5] + __popc(m & ((1u << (pg & 31)) - 1));
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
}
// ... and their rows; the former by a kernel of its own where that is much (see
// mla_table_entries_kernel).
__global__ void __launch_bounds__(256) mla_compact_entries_kernel(const __grid_constant__ CompactParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  compact_entries(p, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}
__global__ void __launch_bounds__(256, kMoveCtas) mla_compact_apply_kernel(const __grid_constant__ CompactParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  if (!p.entries_apart) compact_entries(p, at, step);
  move_pages(p.c, p.ws.head[kHeadMoves], at, step,
             [&](int64_t i, bool) { return make_int2(p.ws.from[i], p.ws.list[i]); });
}

// Up to kLocalPages pages: each CTA decides for itself, in shared memory, and
// moves its share, in one launch.  Counts that are rewritten in place are left
// to the CTA that has read them last, found by a ticket that it sets back to 0.
constexpr int kLocalThreads = 256;
struct CompactLocal {
  Scan<1, int32_t, kLocalThreads> scan;
  int32_t last;
  int32_t pre[kLocalPages / 32];
  union {
    uint8_t bytes[kLocalPages / 8];  // a bit a page: in use
    uint32_t words[kLocalPages / 32];
  } mask;
  uint16_t list[kLocalPages / 2], from[kLocalPages / 2];
};
__global__ void __launch_bounds__(kLocalThreads, kMoveCtas)
    mla_compact_local_kernel(const __grid_constant__ CompactParams p) {
  __shared__ CompactLocal s;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int tid = threadIdx.x, pages = p.c.num_pages, words = (pages + 31) / 32;
#pragma unroll 4
  for (int base = 0; base < pages; base += 4 * kLocalThreads) {
    const int4 v = four_counts(p.refs_in, base + 4 * tid, pages, 0);
    put_nibble(s.mask.bytes, base / 4 + tid,
               (uint32_t)(v.x > 0) | (uint32_t)(v.y > 0) << 1 | (uint32_t)(v.z > 0) << 2 | (uint32_t)(v.w > 0) << 3);
  }
  __syncthreads();
  if (tid == 0) s.last = p.refs_in == p.refs_out ? atomicAdd(p.ws.head + kHeadTicket, 1) : 0;  // (all has been read)
  // two words a thread
  const uint32_t m0 = 2 * tid < words ? s.mask.words[2 * tid] : 0u;
  const uint32_t m1 = 2 * tid + 1 < words ? s.mask.words[2 * tid + 1] : 0u;
  int32_t v[1] = {__popc(m0) + __popc(m1)}, sum[1];
  s.scan.run(v, sum);
  const int L = sum[0];
  s.pre[2 * tid] = v[0];
  s.pre[2 * tid + 1] = v[0] + __popc(m0);
  __syncthreads();
  auto rank = [&](int pg, bool& used) {  // pages in use before page pg, and whether pg is
    const uint32_t m = s.mask.words[pg >> 5];
    used = m >> (pg & 31) & 1;
    return s.pre[pg >> 5] + __popc(m & ((1u << (pg & 31)) - 1));
  };
  bool unused;
  const int kept = L < pages ? rank(L, unused) : L, moves = L - kept;
  for (int pg = tid; pg < pages; pg += kLocalThreads) {
    bool used;
    const int before = rank(pg, used);
    if (pg < L && !used) s.list[pg - before] = (uint16_t)pg;
    if (pg >= L && used) s.from[before - kept] = (uint16_t)pg;
  }
  __syncthreads();
  const int at = blockIdx.x * kLocalThreads + tid, step = gridDim.x * kLocalThreads;
  if (at == 0 && p.live) *p.live = L;
  for (int64_t i = at; i < p.num_indices; i += step) {
    int32_t pg = p.idx_in[i];
    if (pg != -1) {
      bool used = false;
      const int before = pg >= 0 && pg < pages ? rank(pg, used) : 0;
      if (!used) {
        pg = -1;
        set_error(p.ws.err, MLA_ERR_DEVICE_INDEX);
      } else if (pg >= L) {
        pg = s.list[before - kept];
      }
    }
    p.idx_out[i] = pg;
  }
  if (p.refs_in != p.refs_out) {
    for (int pg = at; pg < pages; pg += step) {
      bool used;
      const int before = rank(pg, used);
      p.refs_out[pg] = pg >= L ? 0 : p.refs_in[used ? pg : s.from[pg - before]];
    }
  } else if (s.last == (int)gridDim.x - 1) {
    // every CTA has read the counts: the holes' first, which come from pages
    // at or above L, then the zeros of those
    for (int i = tid; i < moves; i += kLocalThreads) p.refs_out[s.list[i]] = p.refs_in[s.from[i]];
    __syncthreads();
    for (int pg = L + tid; pg < pages; pg += kLocalThreads) p.refs_out[pg] = 0;
    if (tid == 0) p.ws.head[kHeadTicket] = 0;
  }
  move_pages(p.c, moves, at, step, [&](int64_t i, bool) { return make_int2(s.from[i], s.list[i]); });
}

// The deciding kernel: a cluster of as many CTAs as there are blocks of pages,
// up to kCluster.  Beyond that a kernel of its own goes over the pages first;
// `free_ctas`: the deciding CTAs then need no cluster, and are up to 152.
template <class Kernel, class Params>
cudaError_t plan_launch(Kernel kernel, const int32_t* refs, bool free_ctas, cudaStream_t s, const Params& p) {
  const int blocks = blocks_of(p.c.num_pages);
  if (blocks > kCluster) {
    const MaskParams m{p.ws, refs, p.c.num_pages};
    const cudaError_t e = launch_chained(mla_mask_kernel, (unsigned)blocks, kPlan, s, m);
    if (e != cudaSuccess) return e;
    if (free_ctas) return launch_chained(kernel, (unsigned)(blocks < 152 ? blocks : 152), kPlan, s, p);
  }
  unsigned ctas = 1;
  while ((int)ctas < blocks && ctas < kCluster) ctas *= 2;
  return launch_chained(kernel, ctas, kPlan, s, p, ctas > 1 ? ctas : 0);
}

// CTAs for `threads` threads of work, at most kMaxGrid (the kernels loop).
unsigned grid_for(int64_t threads) {
  const int64_t g = (threads + 255) / 256;
  return (unsigned)(g < 1 ? 1 : (g < kMaxGrid ? g : kMaxGrid));
}
int64_t copy_threads(const PageBytes& c, int64_t pages) {
  return pages * c.num_layers * (kv_segs(c) + scale_segs(c)) * 32;
}
// The scale columns of up to `pages` pages, where they are apart.
template <class Kernel, class Params>
cudaError_t launch_scale_columns(Kernel kernel, int64_t pages, cudaStream_t s, const Params& p) {
  if (!p.c.scale_cols) return cudaSuccess;
  return launch_chained(kernel, grid_for(pages * p.c.num_layers * p.c.page_size), 256, s, p);
}

}  // namespace

cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  const cudaError_t e = launch_chained(mla_copy_pages_kernel, grid_for(copy_threads(p.c, p.n)), 256, s, p);
  return e != cudaSuccess ? e : launch_scale_columns(mla_copy_scale_columns_kernel, p.n, s, p);
}

// The cluster carries a call out by itself where that is little: up to
// kClusterEntries table entries, and at most so many bytes of part-filled pages
// (a fork copies one per sequence; a resize seldom copies any).  Scale columns are
// moved by what the deciding kernel leaves in the workspace.
cudaError_t launch_table(const TableParams& p, cudaStream_t s) {
  // (a page of one row is never part-filled)
  int64_t threads = p.c.page_size == 1 ? 0 : copy_threads(p.c, p.to.batch), entries = p.to.num_indices;
  const int64_t most = threads * 128;  // bytes: 8 units of 16 a thread
  if (!p.forks && entries < p.from.num_indices) entries = p.from.num_indices;
  if (!p.c.scale_cols && p.to.batch <= kPlan && p.c.num_pages <= kLocalPages && entries <= kClusterEntries &&
      most <= (p.forks ? kClusterForkBytes : kClusterResizeBytes))
    return launch_chained(mla_table_local_kernel, kCluster, kPlan, s, p, kCluster);
  cudaError_t e = plan_launch(mla_table_plan_kernel, p.refs, false, s, p);
  if (e != cudaSuccess) return e;
  TableParams q = p;
  q.entries_apart = entries > kApartEntries || threads == 0;
  if (q.entries_apart) {
    e = launch_chained(mla_table_entries_kernel, grid_for(entries), 256, s, q);
    if (e != cudaSuccess || threads == 0) return e;
    e = launch_chained(mla_table_apply_kernel, grid_for(threads), 256, s, q);
    return e != cudaSuccess ? e : launch_scale_columns(mla_table_scale_columns_kernel, p.to.batch, s, q);
  }
  const unsigned by_rows = (grid_for(threads) + 2) / 3, by_entries = grid_for(entries);
  const unsigned quarter = by_rows > by_entries ? by_rows : by_entries;
  e = launch_chained(mla_table_apply_kernel, 4 * (quarter < kMaxGrid / 4 ? quarter : kMaxGrid / 4), 256, s, q);
  return e != cudaSuccess ? e : launch_scale_columns(mla_table_scale_columns_kernel, p.to.batch, s, q);
}

cudaError_t launch_free(int32_t* refs, int32_t num_pages, const int32_t* pages, int32_t n, int32_t* error,
                        cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const FreeParams p{refs, pages, num_pages, n, error};
  return launch_chained(mla_free_kernel, (unsigned)(((int64_t)n + 255) / 256), 256, s, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t s) {
  if (p.c.num_pages <= kLocalPages && !p.c.scale_cols) {
    int64_t threads = copy_threads(p.c, p.c.num_pages / 2);
    if (threads < p.num_indices) threads = p.num_indices;
    const unsigned grid = grid_for(threads);
    return launch_chained(mla_compact_local_kernel, grid < kLocalGrid ? grid : kLocalGrid, kLocalThreads, s, p);
  }
  cudaError_t e = plan_launch(mla_compact_plan_kernel, p.refs_in, true, s, p);
  if (e != cudaSuccess) return e;
  int64_t threads = copy_threads(p.c, p.c.num_pages / 2), entries = p.num_indices;
  if (entries < p.c.num_pages) entries = p.c.num_pages;
  CompactParams q = p;
  q.entries_apart = entries > kApartPages;
  if (q.entries_apart) {
    e = launch_chained(mla_compact_entries_kernel, grid_for(entries), 256, s, q);
    if (e != cudaSuccess) return e;
    entries = 0;
  }
  e = launch_chained(mla_compact_apply_kernel, grid_for(threads < entries ? entries : threads), 256, s, q);
  return e != cudaSuccess ? e : launch_scale_columns(mla_compact_scale_columns_kernel, p.c.num_pages / 2, s, q);
}

}  // namespace mla
