// mla_prompt.cu -- attention of a prompt on the 5th-generation tensor cores
// (include/mla_prompt.h), sm_103a.
//
// A CTA takes one head and up to 256 query tokens of a document, as two tiles of
// 128, and walks the document's keys in tiles of 128 (online softmax):
//   S_g = Q_g K_j^T       128 x 128, k = 192: 12 MMAs of kind::f16, both operands
//                         in shared memory (K-major, 128-byte swizzle)
//   P_g = 2^(S_g c - m)   a thread per row, c = sm_scale log2(e); bf16, written over
//                         the first half of S_g in tensor memory
//   O_g += P_g V_j        128 x 128, k = 128: 8 MMAs, P_g from tensor memory, V_j
//                         MN-major from shared memory as TMA leaves it
// The two tiles alternate: while the softmax warps of one turn S into P, the
// tensor cores work for the other, so neither waits for long.  m is raised (and O,
// l rescaled) only when a row's maximum exceeds it by 2^8.
//
// What a row sees is always a run from the document's first key (causal order, or
// a prefix, whichever is longer, or everything), so the mask is one length per row,
// and key tiles past a query tile's longest run are never loaded.
//
// Bound by the tensor cores for long documents: 640 flop a visible pair and head
// against 2 x 128 exponentials a row and tile.  Shared memory: 96 KB of queries, a
// ring of 8 slots of 16 KB (64 columns x 128 keys: a K tile is three, a V tile two).
// Tensor memory: S_0 S_1 O_0 O_1 of 128 columns each.
#include <cuda.h>
#include <cuda_runtime.h>

#include "mla_common.cuh"
#include "mla_prompt_internal.h"

namespace mla {
namespace {

constexpr int kSlotBytes = 128 * 128;  // 128 rows of 64 bf16 columns
constexpr int kRing = 8;
constexpr int kQChunks = 3, kVChunks = 2, kChunks = kQChunks + kVChunks;
constexpr int kWarps = 10;             // 0-3, 4-7 softmax of tile 0 and 1; 8 copies; 9 MMAs
constexpr float kRaise = 8.f;

struct Smem {
  static constexpr int q = 0;                                  // [2 tiles][3 chunks]
  static constexpr int ring = q + 2 * kQChunks * kSlotBytes;
  static constexpr int bars = ring + kRing * kSlotBytes;
  static constexpr int nbars = 2 * kRing + 2 + 2 + 2 + 2 + 1;
  static constexpr int misc = bars + 8 * nbars;                // tmem base, abort, document
  static constexpr int total = misc + 32;
};
enum { kFull = 0, kEmpty = kRing, kQ = 2 * kRing, kS = kQ + 2, kP = kS + 2, kO = kP + 2, kEnd = kO + 2 };

// TMEM columns
__device__ __forceinline__ uint32_t s_col(int g) { return 128u * g; }
__device__ __forceinline__ uint32_t o_col(int g) { return 256u + 128u * g; }

// kind::f16 instruction descriptor: bf16 A and B, fp32 accumulator, A K-major.
constexpr uint32_t idesc_bf16(int M, int N, int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kIdescS = idesc_bf16(128, 128, 0), kIdescO = idesc_bf16(128, 128, 1), kIdescOHalf = idesc_bf16(128, 64, 1);
constexpr uint64_t kTplK = tc::desc_template(16, 1024, 2);          // K-major, 128-byte swizzle
constexpr uint64_t kTplV = tc::desc_template(kSlotBytes, 1024, 2);  // MN-major: 64-column atoms a slot apart

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// The CTA's share of the batch.
struct Work {
  int q0, k0;       // first rows of the document's tile in the query tensors, of its keys
  int rows;         // query tokens of this CTA (1..256)
  int first;        // the first one's place in the document
  int nq, nk, prefix;
};
// How many keys token i (of the CTA) sees.
__device__ __forceinline__ int seen(const PromptParams& p, const Work& w, int i) {
  if (!p.causal) return w.nk;
  return max(0, min(w.nk, max(w.nk - w.nq + w.first + i + 1, w.prefix)));
}
// Key tiles of query tile g: its last token sees the most.
__device__ __forceinline__ int tiles_of(const PromptParams& p, const Work& w, int g) {
  const int n = min(w.rows - 128 * g, 128);
  return n <= 0 ? 0 : (seen(p, w, 128 * g + n - 1) + kPromptTile - 1) / kPromptTile;
}

// Document b's slots (tiles of 256 tokens) begin at qo_indptr[b] / 256 + b: that is
// at least as many as it has tiles, whatever the lengths, so that no prefix sum
// over the batch is needed.  The document of a slot by a search of 32 probes a
// step.  False: an empty slot.
__device__ __forceinline__ bool find_work(const PromptParams& p, int slot, int lane, Work& w) {
  auto base = [&](int b) { return (__ldg(p.qo_indptr + b) >> 8) + b; };
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
    const int n = __popc(__ballot_sync(0xffffffffu, i < hi && base(i) <= slot));
    lo += n * step;
    hi = min(hi, lo + step);
  }
  const int q = __ldg(p.qo_indptr + lo), qe = __ldg(p.qo_indptr + lo + 1);
  const int k = __ldg(p.kv_indptr + lo), ke = __ldg(p.kv_indptr + lo + 1);
  if (q < 0 || qe < q || qe > p.num_q || k < 0 || ke < k || ke > p.num_kv) return false;  // (reported by another warp)
  const int t = slot - ((q >> 8) + lo);
  w.nq = qe - q;
  w.nk = ke - k;
  if (t < 0 || t > (w.nq - 1) >> 8 || w.nq == 0) return false;
  w.first = kPromptQ * t;
  w.q0 = q + w.first;
  w.k0 = k;
  w.rows = min(kPromptQ, w.nq - w.first);
  w.prefix = p.prefix ? __ldg(p.prefix + lo) : 0;
  return true;
}

struct Ctx {
  uint8_t* smem;
  uint64_t* bar;
  volatile int* abort;
  uint32_t tmem;
  int32_t* err;
  __device__ bool wait(int b, int use) const { return wait_phase(&bar[b], use & 1, abort, err); }
  // by a whole warp, which goes on (or gives up) together
  __device__ bool wait_warp(int b, int use) const { return __all_sync(0xffffffffu, wait(b, use)); }
};

// ------------------------------------------------------------------ copies
__device__ void copies(const PromptParams& p, const Ctx& x, const Work& w, int head, int n0, int n1) {
  const uint64_t keep = policy_evict_last(), once = policy_evict_first();
  for (int g = 0; g < 2; ++g) {
    if ((g ? n1 : n0) == 0) continue;
    mbar_arrive_expect_tx(&x.bar[kQ + g], kQChunks * kSlotBytes);
    uint8_t* dst = x.smem + Smem::q + g * kQChunks * kSlotBytes;
    tma_load_3d(dst, &p.q_nope, 0, head, w.q0 + 128 * g, &x.bar[kQ + g], once);
    tma_load_3d(dst + kSlotBytes, &p.q_nope, 64, head, w.q0 + 128 * g, &x.bar[kQ + g], once);
    tma_load_3d(dst + 2 * kSlotBytes, &p.q_pe, 0, head, w.q0 + 128 * g, &x.bar[kQ + g], once);
  }
  const int n = max(n0, n1);
  int c = 0;
  for (int j = 0; j < n && !*x.abort; ++j) {
    const int row = w.k0 + kPromptTile * j;
    for (int i = 0; i < kChunks; ++i, ++c) {
      const int sl = c % kRing, use = c / kRing;
      if (use >= 1 && !x.wait(kEmpty + sl, use - 1)) break;
      uint64_t* bar = &x.bar[kFull + sl];
      uint8_t* dst = x.smem + Smem::ring + sl * kSlotBytes;
      mbar_arrive_expect_tx(bar, kSlotBytes);
      if (i < 2) tma_load_3d(dst, &p.k_nope, 64 * i, head, row, bar, keep);
      else if (i == 2) tma_load_2d(dst, &p.k_pe, 0, row, bar, keep);
      else tma_load_3d(dst, &p.v, 64 * (i - 3), head, row, bar, keep);
    }
  }
  if (*x.abort) {
    // a wait gave up somewhere: never leave with copies in flight (bounded)
    const uint64_t t0 = global_timer_ns();
    for (int i = 0; i < kRing + 2; ++i) {
      const int armed = i < kRing ? (c + kRing - 1 - i) / kRing : ((i - kRing ? n1 : n0) > 0 ? 1 : 0);
      if (armed == 0) continue;
      uint64_t* bar = i < kRing ? &x.bar[kFull + i] : &x.bar[kQ + i - kRing];
      while (!mbar_try_wait(bar, (armed - 1) & 1) && global_timer_ns() - t0 < kWaitTimeoutNs) {
      }
    }
  }
}

// ------------------------------------------------------------------ MMAs
// One thread, in this order: S_0(0) S_1(0), then for every key tile j O_0(j)
// S_0(j + 1) O_1(j) S_1(j + 1).  MMAs of one thread execute in the order of their
// issue, so S_g(j + 1) may overwrite P_g(j), which O_g(j) read before it.
__device__ void mmas(const Ctx& x, int n0, int n1) {
  const int n = max(n0, n1);
  const uint32_t ring = smem_u32(x.smem + Smem::ring), q = smem_u32(x.smem + Smem::q);
  auto wait_chunks = [&](int j, int from, int to) {
    for (int i = from; i < to; ++i) x.wait(kFull + (kChunks * j + i) % kRing, (kChunks * j + i) / kRing);
  };
  auto release = [&](int j, int from, int to) {
    for (int i = from; i < to; ++i) tc::commit(&x.bar[kEmpty + (kChunks * j + i) % kRing]);
  };
  auto scores = [&](int g, int j) {
    const uint64_t a0 = kTplK + ((q + g * kQChunks * kSlotBytes) >> 4);
#pragma unroll
    for (int c = 0; c < kQChunks; ++c) {
      const uint64_t b0 = kTplK + ((ring + (kChunks * j + c) % kRing * kSlotBytes) >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_ss(x.tmem + s_col(g), a0 + ((c * kSlotBytes + 32 * k) >> 4), b0 + 2 * k, kIdescS, c + k > 0);
    }
    tc::commit(&x.bar[kS + g]);
  };
  auto values = [&](int g, int j) {
    const int s0 = (kChunks * j + kQChunks) % kRing;
    const uint64_t b0 = kTplV + ((ring + s0 * kSlotBytes) >> 4);
    const uint32_t a0 = x.tmem + s_col(g), d = x.tmem + o_col(g);
    if (s0 + 1 < kRing) {
#pragma unroll
      for (int k = 0; k < 8; ++k) mma_ts(d, a0 + 8 * k, b0 + 128 * k, kIdescO, (j > 0) | (k > 0));
    } else {  // the second 64 columns are in the ring's first slot
      const uint64_t b1 = kTplV + (ring >> 4);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        mma_ts(d, a0 + 8 * k, b0 + 128 * k, kIdescOHalf, (j > 0) | (k > 0));
        mma_ts(d + 64, a0 + 8 * k, b1 + 128 * k, kIdescOHalf, (j > 0) | (k > 0));
      }
    }
    tc::commit(&x.bar[kO + g]);
  };
  if (n > 0) {
    wait_chunks(0, 0, kQChunks);
    for (int g = 0; g < 2; ++g) {
      if ((g ? n1 : n0) == 0) continue;
      x.wait(kQ + g, 0);
      if (*x.abort) return;
      tc::fence_after();
      scores(g, 0);
    }
    release(0, 0, kQChunks);
  }
  for (int j = 0; j < n; ++j) {
    wait_chunks(j, kQChunks, kChunks);
    for (int g = 0; g < 2; ++g) {
      const int ng = g ? n1 : n0;
      if (j < ng) {
        x.wait(kP + g, j);
        if (*x.abort) return;
        tc::fence_after();
        values(g, j);
      }
      if (g == 1 || n1 <= j) release(j, kQChunks, kChunks);
      if (j + 1 < ng) {
        wait_chunks(j + 1, 0, kQChunks);
        if (*x.abort) return;
        scores(g, j + 1);
      }
      if (g == 1 || n1 <= j) {
        if (j + 1 < n) release(j + 1, 0, kQChunks);
        break;
      }
    }
  }
}

// ------------------------------------------------------------------ softmax
__device__ void softmax(const PromptParams& p, const Ctx& x, const Work& w, int head, int g, int n) {
  const int ww = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int row = 32 * ww + lane, i = 128 * g + row;  // of the tile, of the CTA
  const bool mine = i < w.rows;
  const int lim = mine ? seen(p, w, i) : 0;
  const uint32_t lanes = x.tmem + ((uint32_t)(32 * ww) << 16);
  const uint32_t ts = lanes + s_col(g), to = lanes + o_col(g);
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    if (!x.wait_warp(kS + g, j)) break;
    tc::fence_after();
    float s[128];
#pragma unroll
    for (int c = 0; c < 4; ++c) tc::ld32(ts + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));
    tc::wait_ld();
    const int left = lim - kPromptTile * j;  // keys of this tile that the row sees
    if (__any_sync(0xffffffffu, left < kPromptTile)) {
#pragma unroll
      for (int k = 0; k < 128; ++k) s[k] = k < left ? s[k] : -INFINITY;
    }
    float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
    for (int k = 4; k < 128; k += 4) {
      t0 = fmaxf(t0, s[k]);
      t1 = fmaxf(t1, s[k + 1]);
      t2 = fmaxf(t2, s[k + 2]);
      t3 = fmaxf(t3, s[k + 3]);
    }
    const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * p.scale_log2;
    const bool raise = top > m + kRaise;
    if (__any_sync(0xffffffffu, raise)) {
      const float f = !raise ? 1.f : (m == -INFINITY ? 0.f : fast_exp2(m - top));
      if (raise) m = top;
      l *= f;
      if (j > 0) {
        if (!x.wait_warp(kO + g, j - 1)) break;
        tc::fence_after();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tc::ld32(to + 32 * c, o);
          tc::wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
          tc::st32(to + 32 * c, o);
        }
        tc::wait_st();
      }
    }
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    const float mm = m == -INFINITY ? 0.f : -m;
    const float2 m2 = make_float2(mm, mm);
    float l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t pk[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float2 e = fma2(make_float2(s[64 * h + 2 * k], s[64 * h + 2 * k + 1]), c2, m2);
        const float a = fast_exp2(e.x), b = fast_exp2(e.y);
        l0 += a;
        l1 += b;
        pk[k] = pack_bf16x2(a, b);
      }
      tc::st32(ts + 32 * h, pk);
    }
    l += l0 + l1;
    const int valid = w.nk - kPromptTile * j;  // keys of the document in this tile
    if (valid < kPromptTile) {
      // rows past the document's last key hold other rows' data: zeros, so that a
      // weight of 0 cannot meet a value that is not finite
      const int c0 = kChunks * j + kQChunks;
      x.wait(kFull + c0 % kRing, c0 / kRing);
      x.wait(kFull + (c0 + 1) % kRing, (c0 + 1) / kRing);
      if (row >= valid) {
#pragma unroll
        for (int c = 0; c < kVChunks; ++c) {
          uint4* dst = reinterpret_cast<uint4*>(x.smem + Smem::ring + (c0 + c) % kRing * kSlotBytes + row * 128);
#pragma unroll
          for (int u = 0; u < 8; ++u) dst[u] = make_uint4(0, 0, 0, 0);
        }
      }
      tc::fence_proxy_async();
    }
    tc::wait_st();
    tc::fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&x.bar[kP + g]);
  }
  if (n > 0 && !x.wait_warp(kO + g, n - 1)) return;
  tc::fence_after();
  const float inv = l > 0.f ? __frcp_rn(l) : (l == 0.f ? 0.f : l);
  uint4* out = reinterpret_cast<uint4*>(p.out + (int64_t)(w.q0 + i) * p.out_token_stride + (int64_t)head * p.out_head_stride);
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t o[32];
    if (n > 0) {
      tc::ld32(to + 32 * c, o);
      tc::wait_ld();
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        y[k] = inv == 0.f ? 0u
                          : pack_bf16x2(__uint_as_float(o[8 * u + 2 * k]) * inv, __uint_as_float(o[8 * u + 2 * k + 1]) * inv);
      if (mine) out[4 * c + u] = make_uint4(y[0], y[1], y[2], y[3]);
    }
    __syncwarp();
  }
  if (mine && p.lse) p.lse[(int64_t)(w.q0 + i) * p.heads + head] = l == 0.f ? -INFINITY : (m + fast_log2(l)) * kLn2;
}

__global__ void __launch_bounds__(32 * kWarps, 1) mla_prompt_kernel(const __grid_constant__ PromptParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* misc = reinterpret_cast<int*>(smem + Smem::misc);
  Ctx x;
  x.smem = smem;
  x.bar = reinterpret_cast<uint64_t*>(smem + Smem::bars);
  x.abort = misc + 1;
  x.err = p.ws_err;
  if (threadIdx.x == 0) {
    for (int i = 0; i < Smem::nbars; ++i) mbar_init(&x.bar[i], i == kP || i == kP + 1 ? 4 : 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  // the last tiles of a document see the most keys: they go first
  const int head = (int)blockIdx.x % p.heads, slot = p.slots - 1 - (int)blockIdx.x / p.heads;
  Work w;
  const bool any = find_work(p, slot, lane, w);
  if (blockIdx.x == 0) {
    // documents that do not fit are reported once
    bool bad = false;
    for (int b = threadIdx.x; b < p.batch; b += 32 * kWarps) {
      const int q = p.qo_indptr[b], qe = p.qo_indptr[b + 1], k = p.kv_indptr[b], ke = p.kv_indptr[b + 1];
      bad |= q < 0 || qe < q || qe > p.num_q || k < 0 || ke < k || ke > p.num_kv;
    }
    if (bad) atomicCAS(p.ws_err, 0, kErrDeviceIndex);
  }
  if (!any) return;  // (every warp finds the same)
  __syncwarp();
  if (warp == 9) {
    tc::alloc(reinterpret_cast<uint32_t*>(misc), 512);
    tc::relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  x.tmem = *reinterpret_cast<uint32_t*>(misc);
  const int n0 = tiles_of(p, w, 0), n1 = tiles_of(p, w, 1);
  if (warp < 8) {
    softmax(p, x, w, head, warp >> 2, warp < 4 ? n0 : n1);
  } else if (warp == 8) {
    if (lane == 0) copies(p, x, w, head, n0, n1);
  } else if (lane == 0) {
    mmas(x, n0, n1);
    // every MMA is complete before tensor memory is given back
    tc::commit(&x.bar[kEnd]);
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(&x.bar[kEnd], 0) && global_timer_ns() - t0 < kWaitTimeoutNs) {
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 9) tc::dealloc(x.tmem, 512);
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& p, cudaStream_t stream) {
  static_assert(Smem::total <= 232448, "shared memory of a CTA");
  cudaError_t e = smem_opt_in<mla_prompt_kernel>(Smem::total);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.slots * p.heads));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = Smem::total;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_prompt_kernel, p);
}

}  // namespace mla
