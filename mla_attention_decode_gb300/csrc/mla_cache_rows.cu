// mla_cache_rows.cu -- rows of the latent cache written, read back and found
// (include/mla_cache.h): mla_cache_append, mla_cache_gather, mla_cache_slots.
#include <type_traits>

#include <cuda_runtime.h>

#include "mla_cache_internal.h"
#include "mla_ptx.cuh"

namespace mla {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void set_error(int32_t* error, int32_t code) {
  if (error) *error = code;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Two fp32 operations an instruction, each rounded as the single one is.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
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
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// The larger of two values, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ void unpack_bf16x8(uint4 r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Eight floats -> eight e2m1 codes (nearest, ties to even, saturating at 6),
// element 2i in the low nibble of byte i.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

__device__ __forceinline__ uint8_t pack_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 a;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tmov.b32 %0, {a, a, a, a};\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return (uint8_t)r;
}

// Four packed bytes (eight e2m1 codes) -> eight floats, exactly.
__device__ __forceinline__ void unpack_e2m1x8(uint32_t r, float (&x)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(r));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// The e8m0 byte of a block with largest magnitude amax: e + 127 for the smallest
// 2^e with amax <= 6 * 2^e = 1.5 * 2^(e + 2), read off amax's own exponent and
// fraction (no logarithm, so exact at every border), and the factor 2^-e.
// All-zero block: 127 (2^0).  Infinity or NaN in the block: 255 (NaN), factor 0.
__device__ __forceinline__ uint32_t e8m0_of(float amax, float& inv) {
  const uint32_t bits = __float_as_uint(amax);
  if (bits == 0) {
    inv = 1.f;
    return 127;
  }
  if (bits >= 0x7f800000u) {
    inv = 0.f;
    return 255;
  }
  int e = (int)(bits >> 23) - 127 - 2 + ((bits & 0x7fffffu) > 0x400000u);
  e = max(e, -127);  // amax < 2^-125 (subnormal amax too): 6 * 2^-127 holds it
  inv = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-126 .. 2^127
  return (uint32_t)(e + 127);
}

// ---------------------------------------------------------------- append
// Bound by bytes at many tokens (a key row's 1152 in and 1152, 576 or 306 out, a
// query head's 128 or 1152 each way), by a chain of three reads (slot or
// position, row, store) at few: 2.1 us a call at 4 tokens into bf16 or e4m3, 2.3 into
// MXFP4, of which an empty launch is 1.2.  7147 tokens with their queries'
// position columns (40 to 46 MB): 9.4, 8.9 and 8.9 us into bf16, e4m3 and MXFP4;
// the arithmetic is paired (two fp32 operations an instruction) since
// instructions were 60% of the issue slots there: 10.0, 10.4 and 9.8 us before.
// A warp holds a row or head as 16 latent columns a lane (8 lane + j and 256 +
// 8 lane + j: each load is a warp-wide run of 512 bytes) and the position columns
// 2 lane and 2 lane + 1.
struct Weights {  // of one lane's columns; 1 where the part has none
  float lat[2][8], pe[2];
};
__device__ __forceinline__ void load_weights8(const void* w, bool fp32, int c, float (&y)[8]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = 1.f;
  } else if (fp32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
    const float4 a = f[0], b = f[1];
    y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w, y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
  } else {
    unpack_bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c), y);
  }
}
__device__ __forceinline__ void load_weights_lat(const mla_norm& n, int part, int lane, Weights& w) {
  if (!(n.apply >> part & 1)) return;
  load_weights8(n.weight[part], n.weight_fp32, 8 * lane, w.lat[0]);
  load_weights8(n.weight[part], n.weight_fp32, 256 + 8 * lane, w.lat[1]);
}
__device__ __forceinline__ void load_weights_pe(const mla_norm& n, int part, int lane, Weights& w) {
  if (!(n.apply >> part & 1)) return;
  const void* p = n.weight[part];
  w.pe[0] = w.pe[1] = 1.f;
  if (p && n.weight_fp32) {
    const float2 f = static_cast<const float2*>(p)[lane];
    w.pe[0] = f.x, w.pe[1] = f.y;
  } else if (p) {
    const uint32_t u = static_cast<const uint32_t*>(p)[lane];
    w.pe[0] = __uint_as_float(u << 16), w.pe[1] = __uint_as_float(u & 0xffff0000u);
  }
}

// y = x / sqrt(mean(x^2) + eps) * w over the 512 latent columns.
__device__ __forceinline__ void norm_lat(const mla_norm& n, int part, const Weights& w, float (&x)[2][8]) {
  if (!(n.apply >> part & 1)) return;
  float2 ss = both(0.f);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 v = make_float2(x[h][j], x[h][j + 1]);
      ss = fma2(v, v, ss);
    }
  const float r = rsqrtf(warp_sum(ss.x + ss.y) * (1.f / kLat) + n.eps);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 v = mul2(mul2(make_float2(x[h][j], x[h][j + 1]), both(r)), make_float2(w.lat[h][j], w.lat[h][j + 1]));
      x[h][j] = v.x;
      x[h][j + 1] = v.y;
    }
}

// The rotation as this lane applies it: column 2 lane + k becomes
// x_k c[k] + partner_k s[k], the sign folded into s.
struct Turn {
  float c[2], s[2];
};
// The turn count pos * inv_freq / 2 pi matters modulo 1 only: with inv_freq / 2 pi
// in units of 2^-64 turns the 64-bit product wraps to exactly that, at any
// position.  Its top 32 bits leave 2^-33 turns, their conversion to fp32 up to
// 2^-26 turns (2^-23.3 radians), sincospi 2 ulp; the plan's own rounding of
// inv_freq / 2 pi (2^-52.4 of it) counts as often as the position says.
// Lane i finds pair i's angle; paired halves (i, i + 32) then fetch the two pairs
// that their columns belong to.
__device__ __forceinline__ Turn turn_of(const AppendParams& p, int t, int lane) {
  Turn r = {{1.f, 1.f}, {0.f, 0.f}};
  if (p.rope.num_axes == 0) return r;
  // through the parameter's address, not the constant bank: each lane reads an
  // entry of its own, which the constant cache would serve one lane at a time
  uint64_t step;
  uint32_t axis;
  asm("ld.u64 %0, [%1];" : "=l"(step) : "l"(&p.rope.turn[lane]));
  asm("ld.u8 %0, [%1];" : "=r"(axis) : "l"(&p.rope.axis[lane]));
  const int64_t pos = p.a.positions[(int64_t)t * p.a.position_stride + axis];
  const uint64_t turns = (uint64_t)pos * step + 0x80000000ull;
  float c, s;
  sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
  c *= p.rope.scale;
  s *= p.rope.scale;
  if (p.rope.interleaved) {
    r.c[0] = r.c[1] = c;
    r.s[0] = -s;
    r.s[1] = s;
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int pair = (2 * lane + k) & 31;
      r.c[k] = __shfl_sync(kFull, c, pair);
      const float sk = __shfl_sync(kFull, s, pair);
      r.s[k] = lane < 16 ? -sk : sk;
    }
  }
  return r;
}

// How the position columns turn: not at all (nothing is multiplied: an infinity
// would make its partner NaN), by pairs (2i, 2i + 1), by pairs (i, i + 32).
enum { kStill = 0, kPairs2 = 1, kHalves = 2 };
__device__ __forceinline__ int turn_kind(const AppendParams& p) {
  return p.rope.num_axes == 0 ? kStill : (p.rope.interleaved ? kPairs2 : kHalves);
}
// The lane's two position columns (`u`: their bf16 pair) normed and rotated.
template <int kNorm, int kTurn>
__device__ __forceinline__ float2 turned_pe(float eps, const Weights& w, const Turn& r, uint32_t u) {
  float2 x = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  if (kNorm) {
    const float q = rsqrtf(warp_sum(fmaf(x.x, x.x, x.y * x.y)) * (1.f / kPe) + eps);
    x = mul2(mul2(x, both(q)), make_float2(w.pe[0], w.pe[1]));
  }
  if (kTurn == kStill) return x;
  float2 y = make_float2(x.y, x.x);  // the partners of columns 2 lane, 2 lane + 1
  if (kTurn == kHalves) y = make_float2(__shfl_xor_sync(kFull, x.x, 16), __shfl_xor_sync(kFull, x.y, 16));
  return fma2(x, make_float2(r.c[0], r.c[1]), mul2(y, make_float2(r.s[0], r.s[1])));
}
// f with the call's norm and turn as constants, so that a loop over heads has no
// branch in it.
template <int k>
using Const = std::integral_constant<int, k>;
template <class F>
__device__ __forceinline__ void by_kind(bool norm, int turn, F f) {
  if (norm) {
    if (turn == kPairs2) f(Const<1>(), Const<kPairs2>());
    else if (turn == kHalves) f(Const<1>(), Const<kHalves>());
    else f(Const<1>(), Const<kStill>());
  } else {
    if (turn == kPairs2) f(Const<0>(), Const<kPairs2>());
    else if (turn == kHalves) f(Const<0>(), Const<kHalves>());
    else f(Const<0>(), Const<kStill>());
  }
}

// One key row into row `slot` of the cache, in its format (sc: the scale of an
// e4m3 cache).
template <int kDtype>
__device__ __forceinline__ void store_row(const AppendParams& p, int32_t slot, float sc, const float (&lat)[2][8],
                                          float2 pe, int lane) {
  if (kDtype == MLA_KV_BF16) {
    uint8_t* dst = p.cache.kv + (int64_t)slot * (2 * kRow);
#pragma unroll
    for (int h = 0; h < 2; ++h) reinterpret_cast<uint4*>(dst)[32 * h + lane] = pack_bf16x8(lat[h]);
    reinterpret_cast<uint32_t*>(dst + 2 * kLat)[lane] = pack_bf16x2(pe.x, pe.y);
  } else if (kDtype == MLA_KV_FP8_E4M3) {
    // e4m3 of the rounded quotient y / scale (not of a product with the reciprocal,
    // which lands on the other side of some borders).  Markstein's correction
    // (P. W. Markstein, IBM J. Res. Dev. 34, 1990): with r the rounded reciprocal of
    // b and q = a r, q less (q b - a) r is a / b rounded.  His proof wants q within
    // one ulp, and a r can be 1.5 off; but only quotients next to a border of e4m3
    // matter here, and there the result is the division's for every 24-bit b (2^23
    // divisors, 16 border fractions, the 7 dividends nearest each: 939 million, all
    // equal).  That holds while nothing over- or underflows: a scale within 2^+-60
    // and quotients below 1024 (past 448 all saturate); what is smaller than 2^-10
    // becomes a zero of y's sign either way (q b - a rather than a - q b: of a zero
    // it is +0, and -0 less +0 is -0).  Else the division itself.  (Dividing each of
    // a lane's 18 columns took 200 of 493 instructions a row.)
    const float r = __frcp_rn(sc);
    float2 q[9], top = both(0.f);
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      const float2 y = i < 8 ? make_float2(lat[i >> 2][2 * (i & 3)], lat[i >> 2][2 * (i & 3) + 1]) : pe;
      const float2 q0 = mul2(y, both(r));
      top = make_float2(max_nan(top.x, fabsf(q0.x)), max_nan(top.y, fabsf(q0.y)));
      q[i] = fma2(fma2(q0, both(sc), make_float2(-y.x, -y.y)), both(-r), q0);
    }
    const bool plain = max_nan(top.x, top.y) < 1024.f && sc > 0x1p-60f && sc < 0x1p60f;
    if (!plain) {
#pragma unroll
      for (int i = 0; i < 9; ++i) {
        const float2 y = i < 8 ? make_float2(lat[i >> 2][2 * (i & 3)], lat[i >> 2][2 * (i & 3) + 1]) : pe;
        q[i] = make_float2(__fdiv_rn(y.x, sc), __fdiv_rn(y.y, sc));
      }
    }
    uint8_t* dst = p.cache.kv + (int64_t)slot * kRow;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = f32x2_to_e4m3x2(q[4 * h + j].x, q[4 * h + j].y);
      reinterpret_cast<uint2*>(dst)[32 * h + lane] = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
    reinterpret_cast<uint16_t*>(dst + kLat)[lane] = (uint16_t)f32x2_to_e4m3x2(q[8].x, q[8].y);
  } else {
    uint8_t* dst = p.cache.kv + (int64_t)slot * (kRow / 2);
    uint8_t* sdst = static_cast<uint8_t*>(p.cache.scale) + (int64_t)slot * p.cache.scale_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // a block of 32 columns: four lanes
      float m = fabsf(lat[h][0]);
#pragma unroll
      for (int j = 1; j < 8; ++j) m = max_nan(m, fabsf(lat[h][j]));
      m = max_nan(m, __shfl_xor_sync(kFull, m, 1));
      m = max_nan(m, __shfl_xor_sync(kFull, m, 2));
      float inv, y[8];
      const uint32_t byte = e8m0_of(m, inv);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 v = mul2(make_float2(lat[h][j], lat[h][j + 1]), both(inv));
        y[j] = v.x;
        y[j + 1] = v.y;
      }
      reinterpret_cast<uint32_t*>(dst)[32 * h + lane] = byte == 255 ? 0u : pack_e2m1x8(y);
      if ((lane & 3) == 0) sdst[8 * h + (lane >> 2)] = (uint8_t)byte;
    }
    // the position columns: two blocks of sixteen lanes
    float m = max_nan(fabsf(pe.x), fabsf(pe.y));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, o));
    float inv;
    const uint32_t byte = e8m0_of(m, inv);
    dst[kLat / 2 + lane] = byte == 255 ? 0 : pack_e2m1x2(pe.x * inv, pe.y * inv);
    if ((lane & 15) == 0) sdst[16 + (lane >> 4)] = (uint8_t)byte;
  }
}

// One warp per key row, or per kHeads query heads of a token, all of whose
// columns are in flight before the first is used, in CTAs of kAppendWarps warps.
// kQ: 0 no queries, 1 their position columns (kHeads 16: the angles once per
// token; 4 heads a warp were no faster at any count, 2.8 against 2.7 us at 64
// tokens and 7.8 against 5.5 at 4096), 2 their latent columns too (kHeads 2).
// 8190 tokens into bf16 with every norm and whole queries (321 MB): 90.5 us with
// a warp per head and the rotation table read from the constant bank, 54.5 with
// 4 heads a warp and CTAs of 8 warps, 52.1 with 2 heads, 50.5 with CTAs of 4 warps
// (2: 50.6, 1: 75.8), 49.7 with the keys' CTAs among the queries': 95% of the copy
// rate.
constexpr int kAppendWarps = 4;
template <int kDtype, int kQ, int kHeads>
__global__ void __launch_bounds__(32 * kAppendWarps) mla_append_kernel(const __grid_constant__ AppendParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // CTAs come in groups of kAppendWarps tokens: one for the keys (if any), kGroups
  // for the queries, so that both kinds of traffic are in flight together
  constexpr int kGroups = kQ ? kQueryHeads / kHeads : 0;
  const int keys = p.a.kv_lat ? 1 : 0, group = (int)blockIdx.x / (keys + kGroups);
  const int role = (int)blockIdx.x - group * (keys + kGroups) - keys;  // -1: keys
  Weights w;
  if (role < 0) {
    const int t = group * kAppendWarps + warp;
    if (t >= p.a.num_tokens) return;
    // everything is asked for before the slot is looked at
    const int32_t slot = p.a.slots[t];
    const float scale = kDtype == MLA_KV_FP8_E4M3 ? *static_cast<const float*>(p.cache.scale) : 1.f;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.a.kv_lat) +
                                                      (int64_t)t * p.a.kv_lat_stride);
    const uint4 a = src[lane], b = src[32 + lane];
    const uint32_t u = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.a.kv_pe) +
                                                         (int64_t)t * p.a.kv_pe_stride)[lane];
    load_weights_lat(p.norm, MLA_PART_KV_LAT, lane, w);
    load_weights_pe(p.norm, MLA_PART_KV_PE, lane, w);
    const Turn r = turn_of(p, t, lane);
    if (slot < 0 || slot >= p.cache.rows) {
      if (slot != -1 && lane == 0) set_error(p.error, MLA_ERR_DEVICE_INDEX);
      return;
    }
    float x[2][8];
    unpack_bf16x8(a, x[0]);
    unpack_bf16x8(b, x[1]);
    norm_lat(p.norm, MLA_PART_KV_LAT, w, x);
    float2 y;
    by_kind(p.norm.apply >> MLA_PART_KV_PE & 1, turn_kind(p),
            [&](auto norm, auto turn) { y = turned_pe<norm.value, turn.value>(p.norm.eps, w, r, u); });
    store_row<kDtype>(p, slot, scale, x, y, lane);
    return;
  }
  if (kQ == 0) return;
  const int task = role * kAppendWarps + warp;  // of the group's kGroups * kAppendWarps
  const int t = group * kAppendWarps + task / (kQ ? kGroups : 1), h0 = task % (kQ ? kGroups : 1) * kHeads;
  if (t >= p.a.num_tokens) return;
  const uint16_t* pe = static_cast<const uint16_t*>(p.a.q_pe) + (int64_t)t * p.a.q_pe_token_stride +
                       (int64_t)h0 * p.a.q_pe_head_stride;
  uint8_t* out = static_cast<uint8_t*>(p.a.q_out) + ((int64_t)t * kQueryHeads + h0) * (2 * kRow);
  uint32_t u[kHeads];
  uint4 v[kQ == 2 ? kHeads : 1][2];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) u[h] = reinterpret_cast<const uint32_t*>(pe + h * p.a.q_pe_head_stride)[lane];
  if (kQ == 2) {
    const uint16_t* lat = static_cast<const uint16_t*>(p.a.q_lat) + (int64_t)t * p.a.q_lat_token_stride +
                          (int64_t)h0 * p.a.q_lat_head_stride;
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[h][i] = reinterpret_cast<const uint4*>(lat + h * p.a.q_lat_head_stride)[32 * i + lane];
    load_weights_lat(p.norm, MLA_PART_Q_LAT, lane, w);
  }
  load_weights_pe(p.norm, MLA_PART_Q_PE, lane, w);
  const Turn r = turn_of(p, t, lane);
  by_kind(p.norm.apply >> MLA_PART_Q_PE & 1, turn_kind(p), [&](auto norm, auto turn) {
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      const float2 y = turned_pe<norm.value, turn.value>(p.norm.eps, w, r, u[h]);
      reinterpret_cast<uint32_t*>(out + h * (2 * kRow) + 2 * kLat)[lane] = pack_bf16x2(y.x, y.y);
    }
  });
  if (kQ == 2) {
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      float x[2][8];
      unpack_bf16x8(v[h][0], x[0]);
      unpack_bf16x8(v[h][1], x[1]);
      norm_lat(p.norm, MLA_PART_Q_LAT, w, x);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        reinterpret_cast<uint4*>(out + h * (2 * kRow))[32 * i + lane] = pack_bf16x8(x[i]);
    }
  }
}

// ---------------------------------------------------------------- gather
// Bound by bytes: a row's own (1152, 576 or 306), its slot, 1152 out.  A thread
// takes 8 columns of a row (16 bytes out; 16, 8 or 4 bytes in), the same columns
// of kGatherDeep rows: their slots are loaded together, then their bytes, then
// everything is stored.  247,792 MXFP4 rows (362 MB): 94 us with one row a
// thread, 70 with two, 61.7 with four, 66.9 with eight; 58.3 with four when the
// rows pass the caches as streamed data; 57.4 in CTAs of 2 x 72 threads instead of
// 4 x 72 (1 x 72: 65.9, 8 x 72: 64.8).  That is 93% of the copy rate.
constexpr int kPer = kRow / 8;                      // 72 threads a row
constexpr int kGatherRows = 2;                      // rows of a CTA's pass
constexpr int kGatherThreads = kPer * kGatherRows;
constexpr int kGatherDeep = 4;

template <int kDtype>
__global__ void __launch_bounds__(kGatherThreads) mla_gather_kernel(const __grid_constant__ GatherParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int c = threadIdx.x % kPer;
  const int64_t t0 = (int64_t)blockIdx.x * (kGatherRows * kGatherDeep) + threadIdx.x / kPer;
  int32_t slot[kGatherDeep];
#pragma unroll
  for (int i = 0; i < kGatherDeep; ++i) {
    const int64_t t = t0 + i * kGatherRows;
    slot[i] = t < p.num_rows ? p.slots[t] : -1;
    if (slot[i] >= p.cache.rows || slot[i] < -1) {
      if (c == 0) set_error(p.error, MLA_ERR_DEVICE_INDEX);
      slot[i] = -1;
    }
  }
  uint4 raw[kGatherDeep];  // the row's 16, 8 or 4 bytes, and the block's scale byte
#pragma unroll
  for (int i = 0; i < kGatherDeep; ++i) {
    if (slot[i] < 0) continue;
    const int64_t s = slot[i];
    if (kDtype == MLA_KV_BF16) {
      raw[i] = __ldcs(reinterpret_cast<const uint4*>(p.cache.kv + s * (2 * kRow)) + c);
    } else if (kDtype == MLA_KV_FP8_E4M3) {
      const uint2 r = __ldcs(reinterpret_cast<const uint2*>(p.cache.kv + s * kRow) + c);
      raw[i].x = r.x;
      raw[i].y = r.y;
    } else {
      raw[i].x = __ldcs(reinterpret_cast<const uint32_t*>(p.cache.kv + s * (kRow / 2)) + c);
      raw[i].y = static_cast<const uint8_t*>(p.cache.scale)[s * p.cache.scale_stride + (c >> 2)];
    }
  }
  const float tensor_scale = kDtype == MLA_KV_FP8_E4M3 ? *static_cast<const float*>(p.cache.scale) : 1.f;
#pragma unroll
  for (int i = 0; i < kGatherDeep; ++i) {
    if (slot[i] < 0) continue;
    if (kDtype == MLA_KV_FP8_E4M3) {
      const uint32_t w[4] = {raw[i].x & 0xffffu, raw[i].x >> 16, raw[i].y & 0xffffu, raw[i].y >> 16};
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(e4m3x2_to_h2(w[j]));
        x[2 * j] = f.x * tensor_scale;
        x[2 * j + 1] = f.y * tensor_scale;
      }
      raw[i] = pack_bf16x8(x);
    } else if (kDtype == MLA_KV_MXFP4) {
      const uint32_t byte = raw[i].y;
      // 2^(byte - 127): 2^-127 is subnormal, 255 is NaN
      const float sc = __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255 ? 0x7fc00000u : byte << 23));
      float x[8];
      unpack_e2m1x8(raw[i].x, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= sc;
      raw[i] = pack_bf16x8(x);
    }
    __stcs(reinterpret_cast<uint4*>(p.out + (t0 + i * kGatherRows) * p.out_stride) + c, raw[i]);
  }
}

// ---------------------------------------------------------------- slots
// One thread per token: the sequence by bisection of qo_indptr (staged in shared
// memory up to kSlotsBatch sequences: each step of a bisection in global memory
// is a round trip), then the page of its row.  Whatever the tables hold,
// nothing outside them is read.
constexpr int kSlotsBatch = 2048, kSlotsThreads = 128;

__global__ void __launch_bounds__(kSlotsThreads) mla_slots_kernel(const __grid_constant__ SlotsParams p) {
  __shared__ int32_t s_qo[kSlotsBatch + 1];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int t = blockIdx.x * kSlotsThreads + threadIdx.x, batch = p.table.batch;
  const int32_t* qo = p.qo_indptr;
  if (batch <= kSlotsBatch) {
    for (int i = threadIdx.x; i <= batch; i += kSlotsThreads) s_qo[i] = qo[i];
    __syncthreads();
    qo = s_qo;
  }
  if (t >= p.num_tokens) return;
  const int P = 1 << p.page_shift;
  int32_t slot = -1;
  int64_t row = 0;
  if (batch > 0 && t < qo[batch]) {
    int lo = 0, hi = batch;  // qo[lo] <= t < qo[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (qo[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int64_t first = qo[lo], end = qo[lo + 1];
    const int64_t a = p.table.page_indptr[lo], b = p.table.page_indptr[lo + 1];
    const int32_t last = p.table.last_page_len[lo];
    bool ok = first <= t && t < end && 0 <= a && a <= b && b <= p.table.num_indices;
    int64_t len = 0;
    if (ok && b > a) {
      ok = last >= 1 && last <= P;
      len = (b - a - 1) * P + last;
    }
    if (ok) {
      row = len - (end - first) + (t - first);
      ok = row >= 0;
    }
    if (ok) {
      const int32_t page = p.table.kv_indices[a + (row >> p.page_shift)];
      ok = page >= 0 && page < p.num_pages;
      if (ok) slot = (page << p.page_shift) + (int32_t)(row & (P - 1));
    }
    if (!ok) set_error(p.error, MLA_ERR_DEVICE_INDEX);
  }
  p.slots[t] = slot;
  if (p.rows) p.rows[(int64_t)t * p.row_stride] = (int32_t)row;
}

}  // namespace

namespace {
template <int kDtype, int kQ, int kHeads>
cudaError_t launch_append_as(const AppendParams& p, cudaStream_t s) {
  const int64_t groups = ((int64_t)p.a.num_tokens + kAppendWarps - 1) / kAppendWarps;
  const int ctas = (p.a.kv_lat ? 1 : 0) + (kQ ? kQueryHeads / kHeads : 0);
  return launch_chained(mla_append_kernel<kDtype, kQ, kHeads>, (unsigned)(groups * ctas), 32 * kAppendWarps, s, p);
}
template <int kDtype>
cudaError_t launch_append_to(const AppendParams& p, cudaStream_t s) {
  if (!p.a.q_pe) return launch_append_as<kDtype, 0, 16>(p, s);
  if (p.a.q_lat) return launch_append_as<kDtype, 2, 2>(p, s);
  return launch_append_as<kDtype, 1, 16>(p, s);
}
}  // namespace

cudaError_t launch_append(const AppendParams& p, int kv_dtype, cudaStream_t s) {
  if (p.a.num_tokens == 0 || (!p.a.kv_lat && !p.a.q_pe)) return cudaSuccess;
  switch (kv_dtype) {
    case MLA_KV_BF16: return launch_append_to<MLA_KV_BF16>(p, s);
    case MLA_KV_FP8_E4M3: return launch_append_to<MLA_KV_FP8_E4M3>(p, s);
    default: return launch_append_to<MLA_KV_MXFP4>(p, s);
  }
}

cudaError_t launch_gather(const GatherParams& p, int kv_dtype, cudaStream_t s) {
  if (p.num_rows == 0) return cudaSuccess;
  constexpr int kRows = kGatherRows * kGatherDeep;
  const unsigned grid = (unsigned)(((int64_t)p.num_rows + kRows - 1) / kRows);
  switch (kv_dtype) {
    case MLA_KV_BF16: return launch_chained(mla_gather_kernel<MLA_KV_BF16>, grid, kGatherThreads, s, p);
    case MLA_KV_FP8_E4M3: return launch_chained(mla_gather_kernel<MLA_KV_FP8_E4M3>, grid, kGatherThreads, s, p);
    default: return launch_chained(mla_gather_kernel<MLA_KV_MXFP4>, grid, kGatherThreads, s, p);
  }
}

cudaError_t launch_slots(const SlotsParams& p, cudaStream_t s) {
  if (p.num_tokens == 0) return cudaSuccess;
  return launch_chained(mla_slots_kernel, (unsigned)((p.num_tokens + kSlotsThreads - 1) / kSlotsThreads), kSlotsThreads, s, p);
}

}  // namespace mla
