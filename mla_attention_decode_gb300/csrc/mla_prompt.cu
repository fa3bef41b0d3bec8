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
// tensor cores work for the other, so neither waits for long.  m is the row's maximum
// over its first key tile, raised (and O, l rescaled) only far above it.
//
// What a row sees is always a run from the document's first key (causal order, or
// a prefix, whichever is longer, or everything), so the mask is one length per row,
// and key tiles past a query tile's longest run are never loaded.
//
// Bound by the tensor cores for long documents: 640 flop a visible pair and head
// against 2 x 128 exponentials a row and tile.  Shared memory: 96 KB of queries, a
// ring of 8 slots of 16 KB (64 columns x 128 keys: a K tile is three, a V tile two).
// Tensor memory: S_0 S_1 O_0 O_1 of 128 columns each.
#include <climits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "mla_common.cuh"
#include "mla_prompt_internal.h"

namespace mla {
namespace {

constexpr int kSlotBytes = 128 * 128;  // 128 rows of 64 bf16 columns
constexpr int kRing = 8;
constexpr int kQChunks = 3, kVChunks = 2, kChunks = kQChunks + kVChunks;
constexpr int kSoftWarps = 16;         // 0-7, 8-15: softmax of tile 0 and 1
constexpr int kCopyWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kWarps = kSoftWarps + 2;
// m is raised when a row's maximum exceeds it by 2^24 (P and the sums keep their
// relative precision in bf16 and fp32 whatever their size; O stays below 2^54 max|v|).
constexpr float kRaise = 24.f;

struct Smem {
  static constexpr int q = 0;                                  // [2 tiles][3 chunks]
  static constexpr int ring = q + 2 * kQChunks * kSlotBytes;
  static constexpr int bars = ring + kRing * kSlotBytes;
  static constexpr int nbars = 19;
  static constexpr int meet = bars + 8 * (nbars + 1);          // float [2 tiles][2 halves][128 rows]
  static constexpr int misc = meet + 2 * 2 * 128 * 4;          // tmem base, abort
  static constexpr int total = misc + 32;
};
// mbarriers.  Those of key tile j come in pairs, used by even and odd j in turn.
enum {
  kKFull = 0,  // [2] K tile j copied
  kVFull = 2,  // [2] V tile j copied
  kQ = 4,      // [2 tiles] queries copied
  kS = 6,      // [2 tiles][2] scores written (their K tile read)
  kO = 10,     // [2 tiles][2] products with V added to O (their V tile and weights read)
  kP = 14,     // [2 tiles][2] weights of the even, odd 32 keys written, O rescaled (8 warps)
  kEnd = 18    // the last MMA
};

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

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
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

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Whether any of 64 threads (two warps, named barrier `id`) says so; all have come here.
__device__ __forceinline__ bool any_of_pair(uint32_t id, bool says) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "bar.red.or.pred p, %1, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)says)
      : "memory");
  return r != 0;
}
// Eight 16-byte units a lane, of eight lanes in a row: unit u of lane r goes to lane u,
// place r.
__device__ __forceinline__ void transpose_units(uint32_t (&y)[32], int lane) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (u & d) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t &a = y[4 * u + k], &b = y[4 * (u + d) + k];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, d);
        a = up ? got : a;
        b = up ? b : got;
      }
    }
  }
}
// Unit k to row k of the rows that there are.
__device__ __forceinline__ void put_rows(uint4* dst, int64_t step, int rows, const uint32_t (&y)[32]) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < rows) dst[k * step] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
}
// 16 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// The CTA's share of the batch.
struct Work {
  int q0, k0;       // first rows of the document's tile in the query tensors, of its keys
  int rows;         // query tokens of this CTA (1..256)
  int first;        // the first one's place in the document
  int nq, nk, prefix;
  int skip;         // keys before this CTA's share of them (a multiple of 128)
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

// A document's bounds, and its slots: [at, at + tiles), a slot a tile of 256 tokens.
struct Doc {
  int q, qe, k, ke, prefix, at;
  __device__ __forceinline__ int tiles(const PromptParams& p) const {  // 0: bounds that do not fit (another warp reports them)
    return q >= 0 && qe > q && qe <= p.num_q && k >= 0 && ke >= k && ke <= p.num_kv ? ((qe - q - 1) >> 8) + 1 : 0;
  }
};
__device__ __forceinline__ Doc load_doc(const PromptParams& p, int b) {
  Doc d;
  d.q = __ldg(p.qo_indptr + b);
  d.qe = __ldg(p.qo_indptr + b + 1);
  d.k = __ldg(p.kv_indptr + b);
  d.ke = __ldg(p.kv_indptr + b + 1);
  d.prefix = p.prefix ? __ldg(p.prefix + b) : 0;
  d.at = (d.q >> 8) + b;
  return d;
}
// The last document with key(b) <= x, key not decreasing, by 32 probes a step.
template <class Key>
__device__ __forceinline__ int last_at_most(int batch, int x, int lane, Key key) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
    const int n = __popc(__ballot_sync(0xffffffffu, i < hi && key(i) <= x));
    lo += n * step;
    hi = min(hi, lo + step);
  }
  return lo;
}
// The document of slot x, or of token x; false: of none.  Up to 32 documents are looked at in one
// round of loads, one a lane, and their slots lie one after the other (a scan), so that
// one whose bounds do not fit takes none and hides no other.  Of more, document b's slots begin at
// qo_indptr[b] / 256 + b, which is as many as the documents before it have at least, and
// a search takes the bounds as not decreasing.
template <bool kToken>
__device__ __forceinline__ bool find_doc(const PromptParams& p, int x, int lane, Doc& d) {
  constexpr unsigned all = 0xffffffffu;
  if (p.batch <= 32) {
    const Doc mine = load_doc(p, min(lane, p.batch - 1));
    const int n = lane < p.batch ? mine.tiles(p) : 0;
    int end = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(all, end, o);
      if (lane >= o) end += v;
    }
    const unsigned has = __ballot_sync(all, n > 0 && (kToken ? mine.q <= x && x < mine.qe : end - n <= x && x < end));
    if (has == 0) return false;
    const int b = __ffs(has) - 1;
    d = {__shfl_sync(all, mine.q, b), __shfl_sync(all, mine.qe, b),     __shfl_sync(all, mine.k, b),
         __shfl_sync(all, mine.ke, b), __shfl_sync(all, mine.prefix, b), __shfl_sync(all, end - n, b)};
    return true;
  }
  auto at = [&](int b) { return kToken ? __ldg(p.qo_indptr + b) : (__ldg(p.qo_indptr + b) >> 8) + b; };
  d = load_doc(p, last_at_most(p.batch, x, lane, at));
  const int n = d.tiles(p);
  return n > 0 && (kToken ? d.q <= x && x < d.qe : d.at <= x && x - d.at < n);
}
__device__ __forceinline__ bool find_work(const PromptParams& p, int slot, int lane, Work& w) {
  Doc d;
  if (!find_doc<false>(p, slot, lane, d)) return false;
  w.nq = d.qe - d.q;
  w.nk = d.ke - d.k;
  w.first = kPromptQ * (slot - d.at);
  w.q0 = d.q + w.first;
  w.k0 = d.k;
  w.rows = min(kPromptQ, w.nq - w.first);
  w.prefix = d.prefix;
  w.skip = 0;
  return true;
}
// Whether token t has been attended: a document holds it, and its tile's slot is that
// document's (with bounds that do not fit it may not be).
__device__ __forceinline__ bool attended(const PromptParams& p, int t, int lane) {
  Doc d, of;
  if (!find_doc<true>(p, t, lane, d)) return false;
  const int slot = d.at + ((t - d.q) >> 8);
  if (p.batch <= 32) return slot < p.slots;
  return find_doc<false>(p, slot, lane, of) && of.at == d.at && of.q == d.q;
}

struct Ctx {
  uint8_t* smem;
  uint64_t* bar;
  volatile int* abort;
  uint32_t tmem;
  int32_t* err;
  // Bounded: the clock is read every 1024 tries only (a wait is a step of the chain
  // of scores, softmax and products that the kernel's time consists of).
  __device__ __forceinline__ bool wait(int b, int use) const {
    if (mbar_try_wait(&bar[b], use & 1)) return true;
    uint64_t since = 0;
    for (int tries = 1; !mbar_try_wait(&bar[b], use & 1); ++tries)
      if (tries % 1024 == 0 && (since = look(since)) == kGaveUp) return false;
    return true;
  }
  static constexpr uint64_t kGaveUp = ~0ull;
  __device__ __noinline__ uint64_t look(uint64_t since) const;
  // by a whole warp, which goes on (or gives up) together
  __device__ bool wait_warp(int b, int use) const { return __all_sync(0xffffffffu, wait(b, use)); }
};

// Of a wait that began at `since` (0: its first look): when it began, or kGaveUp
// after kWaitTimeoutNs, or if another thread of the CTA has given up.
__device__ __noinline__ uint64_t Ctx::look(uint64_t since) const {
  if (*abort) return kGaveUp;
  const uint64_t now = global_timer_ns();
  if (since == 0) return now;
  if (now - since <= kWaitTimeoutNs) return since;
  *abort = 1;
  atomicCAS(err, 0, kErrDeviceTimeout);
  return kGaveUp;
}

// ------------------------------------------------------------------ copies
// One lane.  begin() asks for all that needs no wait (it precedes the CTA's first
// barrier), rest() for what is left.
struct Copies {
  const PromptParams& p;
  const Ctx& x;
  const Work& w;
  int head, n0, n1;
  int ks = 0, vs = 0;  // tiles asked for

  __device__ void queries(int g) const {
    if ((g ? n1 : n0) == 0) return;
    const uint64_t once = policy_evict_first();
    mbar_arrive_expect_tx(&x.bar[kQ + g], kQChunks * kSlotBytes);
    uint8_t* dst = x.smem + Smem::q + g * kQChunks * kSlotBytes;
    tma_load_3d(dst, &p.q_nope, 0, head, w.q0 + 128 * g, &x.bar[kQ + g], once);
    tma_load_3d(dst + kSlotBytes, &p.q_nope, 64, head, w.q0 + 128 * g, &x.bar[kQ + g], once);
    tma_load_3d(dst + 2 * kSlotBytes, &p.q_pe, 0, head, w.q0 + 128 * g, &x.bar[kQ + g], once);
  }
  __device__ uint8_t* slot(int j, int c) const { return x.smem + Smem::ring + (kChunks * j + c) % kRing * kSlotBytes; }
  __device__ void keys(int j) {
    const uint64_t keep = policy_evict_last();
    const int row = w.k0 + kPromptTile * j;
    uint64_t* bar = &x.bar[kKFull + (j & 1)];
    mbar_arrive_expect_tx(bar, kQChunks * kSlotBytes);
    tma_load_3d(slot(j, 0), &p.k_nope, 0, head, row, bar, keep);
    tma_load_3d(slot(j, 1), &p.k_nope, 64, head, row, bar, keep);
    tma_load_2d(slot(j, 2), &p.k_pe, 0, row, bar, keep);
    ++ks;
  }
  __device__ void values(int j) {
    const uint64_t keep = policy_evict_last();
    const int row = w.k0 + kPromptTile * j;
    uint64_t* bar = &x.bar[kVFull + (j & 1)];
    mbar_arrive_expect_tx(bar, kVChunks * kSlotBytes);
    tma_load_3d(slot(j, 3), &p.v, 0, head, row, bar, keep);
    tma_load_3d(slot(j, 4), &p.v, 64, head, row, bar, keep);
    ++vs;
  }
  __device__ void begin() {
    const int n = max(n0, n1);
    if (n == 0) return;
    queries(0);
    keys(0);
    queries(1);
    values(0);
    if (n > 1) keys(1);
  }
  __device__ void rest() {
    // what K tile j and V tile j go over: a slot of K and both of V of tile j - 2, two
    // slots of K of tile j - 1
    auto read = [&](int bar, int j) {
      return (j >= n0 || x.wait(bar + (j & 1), j >> 1)) && (j >= n1 || x.wait(bar + 2 + (j & 1), j >> 1));
    };
    const int n = max(n0, n1);
    for (int j = 1; j < n; ++j) {
      if (j >= 2) {
        if (!read(kO, j - 2)) break;
        keys(j);
      }
      if (!read(kS, j - 1)) break;
      values(j);
    }
    // Never leave with copies in flight, whatever gives up, now or later (bounded): the last
    // use of each barrier.  As a rule the block's products wait for the same.
    const uint64_t t0 = global_timer_ns();
    for (int i = 0; i < 6; ++i) {
      const int armed = i < 4 ? ((i < 2 ? ks : vs) + 1 - (i & 1)) / 2 : ((i - 4 ? n1 : n0) > 0 ? 1 : 0);
      if (armed == 0) continue;
      while (!mbar_try_wait(&x.bar[i], (armed - 1) & 1) && global_timer_ns() - t0 < kWaitTimeoutNs) {
      }
    }
  }
};

// ------------------------------------------------------------------ MMAs
// One warp, of which an elected lane issues (the descriptors are the same in every
// lane, so that they stay in uniform registers), in this order: S_0(0) S_1(0), then for
// every key tile j O_0(j) S_0(j + 1) O_1(j) S_1(j + 1).  MMAs of one thread execute in
// the order of their issue, so S_g(j + 1) may overwrite the weights of tile j, which
// O_g(j) read before it; and the query tiles stay half a period apart, one's softmax
// under the other's MMAs.  Descriptors are a constant high word and a low word to
// which addresses / 16 are added.
__device__ void mmas(const Ctx& x, int n0, int n1) {
  const uint32_t ring = smem_u32(x.smem + Smem::ring) >> 4, q = smem_u32(x.smem + Smem::q) >> 4;
  constexpr uint32_t kSlot = kSlotBytes >> 4;
  auto scores = [&](int g, int j) {
    const uint32_t a0 = (uint32_t)kTplK + q + g * kQChunks * kSlot;
#pragma unroll
    for (int c = 0; c < kQChunks; ++c) {
      const uint32_t b0 = (uint32_t)kTplK + ring + (kChunks * j + c) % kRing * kSlot;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_ss(x.tmem + s_col(g), a0 + c * kSlot + 2 * k, b0 + 2 * k, (uint32_t)(kTplK >> 32), kIdescS, c + k > 0);
    }
    tc::commit(&x.bar[kS + 2 * g + (j & 1)]);
  };
  // 16-key steps of the weights: the first, second 32 keys of each 64
  auto values = [&](int g, int j, int part) {
    const uint32_t s0 = (kChunks * j + kQChunks) % kRing;
    const uint32_t b0 = (uint32_t)kTplV + ring + s0 * kSlot;
    const uint32_t a0 = x.tmem + s_col(g), d = x.tmem + o_col(g);
    if (s0 + 1 < kRing) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 4 * (i >> 1) + 2 * part + (i & 1);
        mma_ts(d, a0 + 8 * k, b0 + 128 * k, (uint32_t)(kTplV >> 32), kIdescO, (j > 0) | (part + i > 0));
      }
    } else {  // the second 64 columns are in the ring's first slot
      const uint32_t b1 = (uint32_t)kTplV + ring;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 4 * (i >> 1) + 2 * part + (i & 1);
        mma_ts(d, a0 + 8 * k, b0 + 128 * k, (uint32_t)(kTplV >> 32), kIdescOHalf, (j > 0) | (part + i > 0));
        mma_ts(d + 64, a0 + 8 * k, b1 + 128 * k, (uint32_t)(kTplV >> 32), kIdescOHalf, (j > 0) | (part + i > 0));
      }
    }
    if (part) tc::commit(&x.bar[kO + 2 * g + (j & 1)]);
  };
  const int n = max(n0, n1);
  if (n == 0 || !x.wait_warp(kKFull, 0)) return;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if ((g ? n1 : n0) == 0) continue;
    if (!x.wait_warp(kQ + g, 0)) return;
    tc::fence_after();
    if (tc::elect()) scores(g, 0);
  }
  for (int j = 0; j < n; ++j) {
    if (!x.wait_warp(kVFull + (j & 1), j >> 1)) return;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int ng = g ? n1 : n0;
      if (j >= ng) continue;
      if (!x.wait_warp(kP + 2 * g, j)) return;
      tc::fence_after();
      if (tc::elect()) values(g, j, 0);
      if (!x.wait_warp(kP + 2 * g + 1, j)) return;
      tc::fence_after();
      if (tc::elect()) values(g, j, 1);
      if (j + 1 < ng) {
        if (!x.wait_warp(kKFull + ((j + 1) & 1), (j + 1) >> 1)) return;
        if (tc::elect()) scores(g, j + 1);
      }
    }
  }
}

// ------------------------------------------------------------------ softmax
// Two warps a 32-row quarter of a tile: warp `half` has its columns [64 half, +64), so
// that each SM sub-partition has four warps to choose from.  The two meet at a barrier
// once a key tile, which tells whether any of them has to raise its maximum: only
// then do they exchange maxima.  No wait is left early: a warp that gives up
// (abort) still comes to every meeting.
__device__ void softmax(const PromptParams& p, const Ctx& x, const Work& w, int head, int split, int g, int n) {
  const int half = (threadIdx.x >> 7) & 1, ww = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int row = 32 * ww + lane, i = 128 * g + row;  // of the tile, of the CTA
  const bool mine = i < w.rows;
  const int lim = mine ? seen(p, w, i) - w.skip : INT_MAX;  // (what rows of no token hold is not written)
  const uint32_t lanes = x.tmem + ((uint32_t)(32 * ww) << 16);
  const uint32_t ts = lanes + s_col(g), to = lanes + o_col(g) + 64 * half;
  float* const meet = reinterpret_cast<float*>(x.smem + Smem::meet) + 256 * g + row;  // + 128 per half
  const uint32_t pair = 1 + 4 * g + ww;                                              // named barrier of the two
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    x.wait_warp(kS + 2 * g + (j & 1), j >> 1);
    tc::fence_after();
    float s[64];
#pragma unroll
    for (int c = 0; c < 2; ++c) tc::ld32(ts + 64 * half + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));
    tc::wait_ld();
    const int left = lim - kPromptTile * j - 64 * half;  // of these 64 keys, those that the row sees
    if (__any_sync(0xffffffffu, left < 64)) {
#pragma unroll
      for (int k = 0; k < 64; ++k) s[k] = k < left ? s[k] : -INFINITY;
    }
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = max3(s[k], s[4 + k], s[8 + k]);
#pragma unroll
    for (int k = 12; k < 60; k += 8)
#pragma unroll
      for (int u = 0; u < 4; ++u) t[u] = max3(t[u], s[k + u], s[k + 4 + u]);
    const float most = fmaxf(max3(t[0], s[60], s[61]), max3(max3(t[1], t[2], t[3]), s[62], s[63]));
    // from here on both have their scores in registers (the weights go over them)
    if (any_of_pair(pair, most * p.scale_log2 > m + kRaise)) {
      meet[128 * half] = most;
      named_bar_sync(pair, 64);
      const float top = fmaxf(most, meet[128 * (half ^ 1)]) * p.scale_log2;
      const bool raise = top > m + kRaise;
      const float f = !raise ? 1.f : (m == -INFINITY ? 0.f : fast_exp2(m - top));
      if (raise) m = top;
      l *= f;
      if (j > 0) {
        x.wait_warp(kO + 2 * g + ((j - 1) & 1), (j - 1) >> 1);
        tc::fence_after();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[16];
          ld16(to + 16 * c, o);
          tc::wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
          st16(to + 16 * c, o);
        }
      }
    }
    const int valid = w.nk - w.skip - kPromptTile * j;  // keys of the document in this tile
    if (valid < kPromptTile) {
      // rows past the document's last key hold other rows' data: zeros, so that a
      // weight of 0 cannot meet a value that is not finite (each half: 64 columns)
      const int c = kChunks * j + kQChunks + half;
      x.wait_warp(kVFull + (j & 1), j >> 1);
      if (row >= valid) {
        uint4* dst = reinterpret_cast<uint4*>(x.smem + Smem::ring + c % kRing * kSlotBytes + row * 128);
#pragma unroll
        for (int u = 0; u < 8; ++u) dst[u] = make_uint4(0, 0, 0, 0);
      }
      tc::fence_proxy_async();
    }
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    const float mm = m == -INFINITY ? 0.f : -m;
    const float2 m2 = make_float2(mm, mm);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t pk[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float2 e = fma2(make_float2(s[32 * h + 2 * k], s[32 * h + 2 * k + 1]), c2, m2);
        e = make_float2(fast_exp2(e.x), fast_exp2(e.y));
        sum = add2(sum, e);
        pk[k] = pack_bf16x2(e.x, e.y);
      }
      st16(ts + 32 * half + 16 * h, pk);
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x.bar[kP + 2 * g + h]);
    }
    l += sum.x + sum.y;
  }
  // the halves' sums (once both have read what they met for last)
  named_bar_sync(pair, 64);
  meet[128 * half] = l;
  named_bar_sync(pair, 64);
  l += meet[128 * (half ^ 1)];
  if (n > 0 && !x.wait_warp(kO + 2 * g + ((n - 1) & 1), (n - 1) >> 1)) return;
  tc::fence_after();
  const float inv = l > 0.f ? __frcp_rn(l) : (l == 0.f ? 0.f : l);
  const float lse = l == 0.f ? -INFINITY : (m + fast_log2(l)) * kLn2;
  // Results leave by runs of 128 bytes of a row: eight lanes' rows change hands by
  // 16-byte units first (a row a lane, each store would touch 32 lines; that took 3700
  // cycles instead of 2400).
  const int r0 = 128 * g + 32 * ww + (lane & 24), unit = lane & 7;  // then: unit `unit` of rows r0..r0 + 7
  const int q0 = w.q0, rows = w.rows;
  const int64_t at = (int64_t)split * p.num_q + q0;
  // (without a key tile O holds anything, and inv is 0)
  if (p.splits > 1) {
    uint4* dst = reinterpret_cast<uint4*>(p.part_o + ((at + r0) * p.heads + head) * MLA_PROMPT_V + 64 * half) + unit;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      uint32_t y[32];
      tc::ld32(to + 32 * c, y);
      tc::wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) y[k] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(y[k]) * inv);
      transpose_units(y, lane);
      put_rows(dst + 8 * c, (int64_t)p.heads * (MLA_PROMPT_V / 4), rows - r0, y);
    }
  } else {
    uint32_t y[32];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t o[16];
      ld16(to + 16 * c, o);
      tc::wait_ld();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        y[8 * c + k] = inv == 0.f ? 0u : pack_bf16x2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
    }
    transpose_units(y, lane);
    put_rows(reinterpret_cast<uint4*>(p.out + (int64_t)(q0 + r0) * p.out_token_stride + (int64_t)head * p.out_head_stride + 64 * half) + unit,
             p.out_token_stride / 8, rows - r0, y);
  }
  if (i < rows && half == 0) {
    if (p.splits > 1) p.part_lse[(at + i) * p.heads + head] = lse;
    else if (p.lse) p.lse[(int64_t)(q0 + i) * p.heads + head] = lse;
  }
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
  if (threadIdx.x == 32 * kCopyWarp) {
    for (int i = 0; i < Smem::nbars; ++i) mbar_init(&x.bar[i], i >= kP && i < kP + 4 ? 8 : 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  // the last tiles of a document see the most keys: they go first
  const int split = (int)blockIdx.x % p.splits, tile = (int)blockIdx.x / p.splits;
  const int head = tile % p.heads, slot = p.slots - 1 - tile / p.heads;
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
  int n0 = tiles_of(p, w, 0), n1 = tiles_of(p, w, 1);
  if (p.splits > 1) {
    const int n = max(n0, n1), lo = n * split / p.splits, hi = n * (split + 1) / p.splits;
    n0 = max(0, min(n0, hi) - lo);
    n1 = max(0, min(n1, hi) - lo);
    w.skip = kPromptTile * lo;
    w.k0 += w.skip;
  }
  Copies copies{p, x, w, head, n0, n1};
  if (warp == kMmaWarp) {
    tc::alloc(reinterpret_cast<uint32_t*>(misc), 512);
    tc::relinquish();
  } else if (threadIdx.x == 32 * kCopyWarp) {
    copies.begin();
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  x.tmem = *reinterpret_cast<uint32_t*>(misc);
  if (warp < kSoftWarps) {
    softmax(p, x, w, head, split, warp >> 3, warp < 8 ? n0 : n1);
  } else if (warp == kCopyWarp) {
    if (lane == 0) copies.rest();
  } else {
    x.tmem = __shfl_sync(0xffffffffu, x.tmem, 0);
    mmas(x, __shfl_sync(0xffffffffu, n0, 0), __shfl_sync(0xffffffffu, n1, 0));
    // every MMA is complete before tensor memory is given back
    __syncwarp();
    if (tc::elect()) tc::commit(&x.bar[kEnd]);
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(&x.bar[kEnd], 0) && global_timer_ns() - t0 < kWaitTimeoutNs) {
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(x.tmem, 512);
}

// The partial results of a row joined: a warp a token and head, 4 columns a lane.
constexpr int kJoinWarps = 4;
__global__ void __launch_bounds__(32 * kJoinWarps) mla_prompt_join_kernel(const __grid_constant__ PromptParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5), rows = (int64_t)p.num_q * p.heads;
  if (row >= rows) return;
  const int t = (int)(row / p.heads), head = (int)(row - (int64_t)t * p.heads);
  const float mine = lane < p.splits ? p.part_lse[lane * rows + row] : -INFINITY;
  float4 v[kPromptMaxSplits];
#pragma unroll
  for (int s = 0; s < kPromptMaxSplits; ++s)
    if (s < p.splits) v[s] = reinterpret_cast<const float4*>(p.part_o + (s * rows + row) * MLA_PROMPT_V)[lane];
  if (!attended(p, t, lane)) return;  // a row of no document stays as it is (what was read is no result)
  float top = mine;
  bool nan = mine != mine;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  nan = __any_sync(0xffffffffu, nan);
  top = __shfl_sync(0xffffffffu, top, 0);
  const float w = mine == -INFINITY ? 0.f : fast_exp2((mine - top) * kLog2e);
  float sum = w;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  sum = __shfl_sync(0xffffffffu, sum, 0);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int s = 0; s < kPromptMaxSplits; ++s) {
    const float ws = __shfl_sync(0xffffffffu, w, s);
    if (s < p.splits && ws != 0.f) {
      y.x = fmaf(ws, v[s].x, y.x);
      y.y = fmaf(ws, v[s].y, y.y);
      y.z = fmaf(ws, v[s].z, y.z);
      y.w = fmaf(ws, v[s].w, y.w);
    }
  }
  const float inv = nan ? NAN : (sum > 0.f ? __frcp_rn(sum) : 0.f);
  uint2* out = reinterpret_cast<uint2*>(p.out + (int64_t)t * p.out_token_stride + (int64_t)head * p.out_head_stride);
  out[lane] = make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
  if (lane == 0 && p.lse) p.lse[row] = nan ? NAN : (sum > 0.f ? top + fast_log2(sum) * kLn2 : -INFINITY);
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& p, cudaStream_t stream) {
  static_assert(Smem::total <= 232448, "shared memory of a CTA");
  cudaError_t e = smem_opt_in<mla_prompt_kernel>(Smem::total);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.slots * p.heads * p.splits));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = Smem::total;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, mla_prompt_kernel, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)p.num_q * p.heads;
  cfg.gridDim = dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, mla_prompt_join_kernel, p);
}

}  // namespace mla
