// pa_cache4.cuh - quantise-and-write of new K / V rows into the 4-bit paged cache: what
// a warp does with its unit (included by pa_cache4.cu and pa_rope.cu).
//
// A block is 16 neighbouring dims of one position.  With the tensor scale g
// (per kv head, per channel or one for all; fp32) of each element x (bf16):
//   y = x / g, a = max |y| over the block;  s = E4M3(min(a / M, 448)), M = 6
//   (FP4 E2M1) or 7 (int4), round to nearest even;  step = s * g;
//   code = nearest code to x / step, ties to even, saturated at +-M; 0 where
//   step is 0.  Quotients and products are IEEE binary32.
// A NaN is written as 0 and does not count towards a (the cache then holds no
// NaN that a masked position could spread); an infinity saturates its block's
// scale and itself.
//
// One warp per (sequence, unit of 32 or 8 positions of the appended range, kv
// head, K or V), each reading its rows once with coalesced 8- or 16-byte loads:
//   K: lane = 8 dims of one row (two lanes per block), codes leave as a 32-bit
//      word per lane;
//   V: lane = 4 dims of all the unit's positions (four lanes per block), so a
//      dim's code bytes of the unit gather in the lane's registers and leave as
//      one store.
// The block maximum of uniform scales is taken on the bf16 bits, two elements a
// step; the lanes of a block then work out a different row's scale each and
// share them.  Quotients: an approximate reciprocal, and one correction of the
// quotient by its residual, which gives every quotient that is exactly a border
// between two codes exactly, and the others to the last bit.
// Rows that are not aligned and blocks out of the common range (a scale that is
// not a normal E4M3 number or is saturated, infinities, NaN) go position by
// position with divisions.  Where the range covers a unit in part, the nibbles of
// other positions stay (one warp owns a unit, so nobody else writes its bytes).
// What bounds it: 2.56 bytes per element against the quantiser's instructions (quotients by
// pairs): 31k rows of 8 heads in 37.6 us (int4) or 34.6 (FP4), 4.3 and 4.7 TB/s; with
// per-channel scales 63 and 57.  (Requesting the next rows before the current ones are worked
// on spills, and gained nothing.)  That is for blocks of the common range.  A block whose
// max |x / g| is below M / 64 (its scale is subnormal, or 0 for a block of zeros) sends
// the four K rows or the V unit that hold it through the divisions: the same rows times
// 0.03 with g = 1 took 317 us, rows of which every 16th is 0 315.
#pragma once

#include "pa_common.cuh"
#include "pa_kv4.cuh"

namespace pa {
namespace {

struct Append4Params {
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  int64_t kv_stride;
  uint8_t* cache_k;
  uint8_t* cache_v;
  const void* k_scale;
  const void* v_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* seq_lens_kv;
  const int32_t* cu_seqlens_q;
  int32_t* status;
  int32_t max_blocks;
  int32_t num_pages;
  int32_t kv_heads;
  int32_t scale_kind;
  RowUnits units;
  int32_t vec;         // rows may be read with 16-byte loads
  uint32_t total;      // (sequence, unit, kv head, side) warps
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x / d with r close to 1 / d: Markstein's correction of a quotient by its residual,
// which one fused multiply-add gives exactly
__device__ __forceinline__ float quot(float x, float d, float r) {
  const float q = x * r;
  return __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
}

// Pairs of binary32 numbers, an operation of each rounded by itself.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}

// quot() of a pair
__device__ __forceinline__ float2 quot2(float2 x, float2 d, float2 r) {
  const float2 q = mul2(x, r);
  return fma2(fma2(q, make_float2(-d.x, -d.y), x), r, q);
}

// The quotients of two neighbouring dims, as a pair or one by one.
template <bool PAIRS>
__device__ __forceinline__ float2 quot_dims(float2 x, float2 d, float2 r) {
  if constexpr (PAIRS) return quot2(x, d, r);
  else return make_float2(quot(x.x, d.x, r.x), quot(x.y, d.y, r.y));
}

template <bool PAIRS>
__device__ __forceinline__ float2 mul_dims(float2 a, float2 b) {
  if constexpr (PAIRS) return mul2(a, b);
  else return make_float2(a.x * b.x, a.y * b.y);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float2 bf16_2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

template <int FP4>
struct Fmt {
  static constexpr float kTop = FP4 ? 6.0f : 7.0f;
};

// Block scale from max |x / g| / M: the E4M3 byte.
template <int FP4>
__device__ __forceinline__ uint32_t block_scale(float a) {
  uint16_t sb;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.0f), "f"(a));
  return sb & 0xFFu;
}

// Whether the short quotients hold for a block of maximum a = max |x / g|: a
// normal, unsaturated scale and a step far from the ends of the exponent range
// (false for NaN).
template <int FP4>
__device__ __forceinline__ bool common(float a, float s, float step) {
  return s >= 0.015625f && a < 448.0f * Fmt<FP4>::kTop && step > 1e-30f && step < 1e30f;
}

// Eight quotients -> eight codes, the first in the lowest nibble.
template <int FP4>
__device__ __forceinline__ uint32_t pack8(const float (&q)[8]) {
  uint32_t w;
  if constexpr (FP4) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  } else {
    // adding 2^23 + 2^22 + 8 rounds to an integer, ties to even, and leaves code
    // + 8 in the low bits; the words are summed at 4-bit distances and what the
    // constant adds to them is taken off, as is the 8 of every code
    constexpr uint32_t kBits = 0x4B400000u;   // 2^23 + 2^22 as fp32
    uint32_t off = 0;
    w = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      w = (w << 4) + __float_as_uint(q[i] + 12582920.0f);
      off = (off << 4) + kBits;
    }
    w = (w - off) ^ 0x88888888u;
  }
  return w;
}

// ---- any positions, any values: [lo, hi) of the half page, lane = 4 dims
template <int FP4>
__device__ __noinline__ void write_any(const __nv_bfloat16* src, int64_t stride, const void* scale, int kind, int kvh,
                                       uint8_t* half, bool value_side, int lo, int hi, int lane) {
  constexpr float kTop = Fmt<FP4>::kTop;
  float g[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    g[e] = load_scale(scale, kind, kind == PA_SCALE_PER_CHANNEL ? kvh * kV4Dim + 4 * lane + e : kvh);
  src += 4 * lane;
#pragma unroll 1
  for (int r = lo; r < hi; ++r, src += stride) {
    float x[4], a = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = __bfloat162float(src[e]);
      if (x[e] != x[e]) x[e] = 0.0f;
      a = fmaxf(a, fabsf(__fdiv_rn(x[e], g[e])));
    }
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const uint32_t sb = block_scale<FP4>(__fdiv_rn(a, kTop));
    const float s = e4m3_to_f32(sb);
    float q[8] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float step = __fmul_rn(s, g[e]);
      q[e] = fminf(fmaxf(step > 0.0f ? __fdiv_rn(x[e], step) : 0.0f, -kTop), kTop);
    }
    const uint32_t w = pack8<FP4>(q);
    if (value_side) {
      const int sh = 4 * (r & 1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint8_t* v = half + (4 * lane + e) * (kV4Half / 2) + r / 2;
        *v = (uint8_t)((*v & (0xF0u >> sh)) | ((w >> (4 * e)) & 15u) << sh);
      }
      if ((lane & 3) == 0) half[kV4Codes + (lane >> 2) * kV4Half + r] = (uint8_t)sb;
    } else {
      *reinterpret_cast<uint16_t*>(half + r * (kV4Dim / 2) + 2 * lane) = (uint16_t)w;
      if ((lane & 3) == 0) half[kV4Codes + r * kV4Nblk + (lane >> 2)] = (uint8_t)sb;
    }
  }
}

// ---- K, positions [lo, hi) of the unit of U that starts at `first` of the half
// page (FULL: all of them); rows: the row of position lo
template <int FP4, bool PC, int U, bool FULL, bool PAIRS = true>
__device__ __forceinline__ void write_k(const Append4Params& p, const __nv_bfloat16* rows, uint8_t* half, int kvh,
                                        int first, int lo, int hi, int lane) {
  auto in = [&](int r) { return FULL || (r >= lo && r < hi); };
  const int c = lane & 15, r0 = lane >> 4;   // dims 8c .. 8c+7 of rows r0, r0 + 2, ...
  float g[8], rg[8];
#pragma unroll
  for (int e = 0; e < (PC ? 8 : 1); ++e) {
    g[e] = load_scale(p.k_scale, p.scale_kind, PC ? kvh * kV4Dim + 8 * c + e : kvh);
    rg[e] = rcp_approx(g[e]);
  }
  const __nv_bfloat16* src = rows + (FULL ? r0 : r0 - lo) * p.kv_stride + 8 * c;
  const int64_t s2 = 2 * p.kv_stride;
  uint8_t* codes = half + (first + r0) * (kV4Dim / 2) + 4 * c;
  uint8_t* scales = half + kV4Codes + (first + 2 * (lane & 1) + r0) * kV4Nblk + (c >> 1);
#pragma unroll 1
  for (int base = 0; base < U; base += 8) {
    if (!FULL && (base + 8 <= lo || base >= hi)) {
      src += 4 * s2;
      continue;
    }
    uint4 xs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i, src += s2)
      xs[i] = in(base + 2 * i + r0) ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // rows base + 4h + {0, 2} + r0
      const uint4* x = xs + 2 * h;
      float f[2][8];
      uint32_t m[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[i][2 * e] = bf16_lo(w[e]);
          f[i][2 * e + 1] = bf16_hi(w[e]);
        }
        m[i] = max_u16x2(max_u16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                         max_u16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
      }
      // the block maxima of both rows; an even lane goes on with the first row's
      uint32_t mm = max_u16x2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
      mm = max_u16x2(mm, __shfl_xor_sync(0xffffffffu, mm, 1));
      const uint32_t mine = (lane & 1) ? mm >> 16 : mm & 0xFFFFu;
      float a;
      if constexpr (PC) {
        float y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          y[i] = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 v = quot_dims<PAIRS>(make_float2(f[i][e], f[i][e + 1]), make_float2(g[e], g[e + 1]), make_float2(rg[e], rg[e + 1]));
            y[i] = fmaxf(fmaxf(y[i], fabsf(v.x)), fabsf(v.y));
          }
        }
        const float t = (lane & 1) ? y[0] : y[1];
        a = fmaxf((lane & 1) ? y[1] : y[0], __shfl_xor_sync(0xffffffffu, t, 1));
      } else {
        a = quot(__uint_as_float(mine << 16), g[0], rg[0]);
      }
      const uint32_t sb = block_scale<FP4>(quot(a, Fmt<FP4>::kTop, 1.0f / Fmt<FP4>::kTop));
      const float s = e4m3_to_f32(sb), st = PC ? s : s * g[0], rs = rcp_approx(st);
      const bool mine_in = in(base + 4 * h + 2 * (lane & 1) + r0);
      if (__all_sync(0xffffffffu, !mine_in || (mine < 0x7F80u && common<FP4>(a, s, st)))) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float si = __shfl_sync(0xffffffffu, st, (lane & ~1) | i);
          const float ri = __shfl_sync(0xffffffffu, rs, (lane & ~1) | i);
          float q[8];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 s2 = make_float2(si, si), r2 = make_float2(ri, ri);
            const float2 v = quot_dims<PAIRS>(make_float2(f[i][e], f[i][e + 1]),
                                              PC ? mul_dims<PAIRS>(s2, make_float2(g[e], g[e + 1])) : s2,
                                              PC ? mul_dims<PAIRS>(r2, make_float2(rg[e], rg[e + 1])) : r2);
            q[e] = v.x;
            q[e + 1] = v.y;
          }
          if (in(base + 4 * h + 2 * i + r0))
            *reinterpret_cast<uint32_t*>(codes + (base + 4 * h + 2 * i) * (kV4Dim / 2)) = pack8<FP4>(q);
        }
        if (mine_in) scales[(base + 4 * h) * kV4Nblk] = (uint8_t)sb;
      } else {
        const int a0 = FULL ? base + 4 * h : max(lo, base + 4 * h);
        write_any<FP4>(rows + (FULL ? a0 : a0 - lo) * p.kv_stride, p.kv_stride, p.k_scale, p.scale_kind, kvh, half,
                       false, first + a0, first + (FULL ? base + 4 * h + 4 : min(hi, base + 4 * h + 4)), lane);
      }
    }
  }
}

// ---- V, the same: four dims of every position per lane
template <int FP4, bool PC, int U, bool FULL, bool PAIRS = true>
__device__ __forceinline__ void write_v(const Append4Params& p, const __nv_bfloat16* rows, uint8_t* half, int kvh,
                                        int first, int lo, int hi, int lane) {
  auto in = [&](int r) { return FULL || (r >= lo && r < hi); };
  const int sub = lane & 3, blk = lane >> 2;
  float g[4], rg[4];
#pragma unroll
  for (int e = 0; e < (PC ? 4 : 1); ++e) {
    g[e] = load_scale(p.v_scale, p.scale_kind, PC ? kvh * kV4Dim + 4 * lane + e : kvh);
    rg[e] = rcp_approx(g[e]);
  }
  const __nv_bfloat16* src = rows - (FULL ? 0 : lo * p.kv_stride) + 4 * lane;
  uint8_t* scales = half + kV4Codes + blk * kV4Half + first + sub;
  uint32_t out[4][U / 8];   // [dim][8-position word]
  bool all_common = true;
#pragma unroll
  for (int k = 0; k < U / 8; ++k) {
    uint2 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j, src += p.kv_stride)
      x[j] = in(8 * k + j) ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
    float q[4][8];   // [dim][position]
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // positions 4h .. 4h+3; lane `sub` works out the scale of 4h + sub
      uint32_t m[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        m[j] = max_u16x2(x[4 * h + j].x & 0x7FFF7FFFu, x[4 * h + j].y & 0x7FFF7FFFu);
      uint32_t m01 = max_u16x2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
      uint32_t m23 = max_u16x2(__byte_perm(m[2], m[3], 0x5410), __byte_perm(m[2], m[3], 0x7632));
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        m01 = max_u16x2(m01, __shfl_xor_sync(0xffffffffu, m01, o));
        m23 = max_u16x2(m23, __shfl_xor_sync(0xffffffffu, m23, o));
      }
      const uint32_t mp = (sub & 2) ? m23 : m01;
      const uint32_t mine = (sub & 1) ? mp >> 16 : mp & 0xFFFFu;
      float f[4][4];   // [position][dim]
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j][0] = bf16_lo(x[4 * h + j].x);
        f[j][1] = bf16_hi(x[4 * h + j].x);
        f[j][2] = bf16_lo(x[4 * h + j].y);
        f[j][3] = bf16_hi(x[4 * h + j].y);
      }
      float a;
      if constexpr (PC) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 v = quot_dims<PAIRS>(make_float2(f[j][e], f[j][e + 1]), make_float2(g[e], g[e + 1]), make_float2(rg[e], rg[e + 1]));
            y[j] = fmaxf(fmaxf(y[j], fabsf(v.x)), fabsf(v.y));
          }
          y[j] = fmaxf(y[j], __shfl_xor_sync(0xffffffffu, y[j], 1));
          y[j] = fmaxf(y[j], __shfl_xor_sync(0xffffffffu, y[j], 2));
        }
        a = (sub & 2) ? ((sub & 1) ? y[3] : y[2]) : ((sub & 1) ? y[1] : y[0]);
      } else {
        a = quot(__uint_as_float(mine << 16), g[0], rg[0]);
      }
      const uint32_t sb = block_scale<FP4>(quot(a, Fmt<FP4>::kTop, 1.0f / Fmt<FP4>::kTop));
      // (a position out of the range gets finite codes: a word holds several)
      const bool mine_in = in(8 * k + 4 * h + sub);
      const float s = e4m3_to_f32(sb), st = !mine_in ? 1.0f : PC ? s : s * g[0], rs = rcp_approx(st);
      all_common = all_common && (!mine_in || (mine < 0x7F80u && common<FP4>(a, s, st)));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float sj = __shfl_sync(0xffffffffu, st, (lane & ~3) | j);
        const float rj = __shfl_sync(0xffffffffu, rs, (lane & ~3) | j);
        const float2 s2 = make_float2(sj, sj), r2 = make_float2(rj, rj);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 v = quot_dims<PAIRS>(make_float2(f[j][e], f[j][e + 1]),
                                            PC ? mul_dims<PAIRS>(s2, make_float2(g[e], g[e + 1])) : s2,
                                            PC ? mul_dims<PAIRS>(r2, make_float2(rg[e], rg[e + 1])) : r2);
          q[e][4 * h + j] = v.x;
          q[e + 1][4 * h + j] = v.y;
        }
      }
      if (mine_in) scales[8 * k + 4 * h] = (uint8_t)sb;
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) out[d][k] = pack8<FP4>(q[d]);
  }
  uint8_t* dst = half + 4 * lane * (kV4Half / 2) + first / 2;
  if (!__all_sync(0xffffffffu, all_common)) {   // the unit again, codes and scales
    write_any<FP4>(rows, p.kv_stride, p.v_scale, p.scale_kind, kvh, half, true, first + (FULL ? 0 : lo),
                   first + (FULL ? U : hi), lane);
  } else if constexpr (!FULL) {
    // the nibbles of positions out of the range stay
#pragma unroll
    for (int k = 0; k < U / 8; ++k) {
      const int a = max(0, min(8, lo - 8 * k)), b = max(0, min(8, hi - 8 * k));
      const uint32_t mask = (uint32_t)(((1ull << (4 * b)) - 1) & ~((1ull << (4 * a)) - 1));
      if (mask != 0) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t* w = reinterpret_cast<uint32_t*>(dst + d * (kV4Half / 2)) + k;
          *w = mask == 0xFFFFFFFFu ? out[d][k] : (*w & ~mask) | (out[d][k] & mask);
        }
      }
    }
  } else if constexpr (U == 32) {
#pragma unroll
    for (int d = 0; d < 4; ++d)
      reinterpret_cast<uint4*>(dst)[d] = make_uint4(out[d][0], out[d][1], out[d][2], out[d][3]);
  } else {
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int k = 0; k < U / 8; ++k) reinterpret_cast<uint32_t*>(dst + d * (kV4Half / 2))[k] = out[d][k];
  }
}

}  // namespace
}  // namespace pa
