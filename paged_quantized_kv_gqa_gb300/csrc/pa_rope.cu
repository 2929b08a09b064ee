// pa_rope.cu - the step before attention in one launch (two for many rows): queries rotated by their
// positions, new K / V rows rotated (K), quantised and written into the paged cache.
//
// Rotation of a pair (a, b) of dims by the angle whose cos c and sin s the table holds,
// every product and sum rounded to binary32 by itself (no fused multiply-add, so that a
// stored code is a function of the inputs that another program can reproduce):
//   a' = a c - b s,  b' = b c + a s.
// Queries are rounded to bf16 once; K goes to its quantiser in binary32, with the values
// that pa_cache.cu / pa_cache4.cuh write for a row of such numbers:
//   8 bits  Q(x / s); 4 bits  per block of 16 dims e = E4M3(min(max |x / g| / M, 448)),
//   step = e g, code = nearest to x / step.
// V is written as pa_cache_append writes it.
//
// GQA: lane = 8 dims of a row, two rows a step, so that a lane's cos and sin are read
// once for all heads of its row; the other dim of a pair comes by a shuffle (halves) or
// is the lane's own (adjacent).  A warp takes a unit of 2 to 8 positions and a group of the
// heads, the queries' first, K's behind them.  V: a warp per (unit, kv head), lane = 4
// dims of all the unit's positions, whose bytes gather in registers.
// MLA: 8 lanes hold the 64 rotated dims of a head, 4 query heads a step; a latent row is
// one warp's.
#include <algorithm>
#include <cmath>

#include "pa_cache4.cuh"

namespace pa {
namespace {

constexpr int kPage = 64;
constexpr int kWarps = 8;
constexpr int kQCtas = 4;   // CTAs an SM of the queries' kernel
constexpr int kMlaRow = 576, kMlaQ = 192, kMlaNope = 128;

struct RopeParams {
  Append4Params a;             // the rows, cache, scales and lengths (units, total: the V warps')
  const float* cos_sin;
  const int32_t* positions;    // [axes][total_q] or null
  const __nv_bfloat16* q;      // or null
  __nv_bfloat16* q_out;
  int64_t q_stride, q_out_stride;
  RowUnits units;              // the rotation's, of 1 << unit_shift positions
  int32_t unit_shift;
  uint32_t rot_warps;          // warps of the rotation; the V warps follow
  int32_t groups, group_heads; // head groups of a unit
  int32_t q_heads;             // 0 without queries
  int32_t table_rows, rot, adjacent, axes, quads;   // quads: four neighbouring pairs share an axis
  int32_t total_q;
  int32_t k_scale16, v32;      // per-channel K scales are 16-byte, cache_v 32-byte aligned
  uint32_t pair_axis[4];       // two bits a pair
  float neg_zero;              // -0, unknown to the compiler (turn8)
};

__device__ __forceinline__ uint32_t bf16x2_of(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// cos and sin (signed for its place in the pair) of a lane's 8 dims
struct Turn {
  float2 c[4], s[4];
};

// Fills `a` for dims 8 o .. 8 o + 7 of a rotated width of p.rot in row t at position
// pos; false (and the status recorded) when a position is not a row of the table.
__device__ __forceinline__ bool load_turn(const RopeParams& p, int64_t t, int pos, int o, Turn& a) {
  const int half = p.rot / 2;
  // dims 8 o .. are the first of their pairs in the lower half of `halves`
  const int pair0 = p.adjacent ? 4 * o : 8 * o % half;
  int row[4] = {pos, 0, 0, 0};
  if (p.positions != nullptr) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < p.axes) row[k] = __ldg(p.positions + (int64_t)k * p.total_q + t);
  }
  const int axes = p.positions != nullptr ? p.axes : 1;
  bool ok = true;
#pragma unroll
  for (int k = 0; k < 4; ++k) ok = ok && (k >= axes || (row[k] >= 0 && row[k] < p.table_rows));
  if (!ok) {
    record_status(p.a.status, PA_ERR_BAD_POSITION, (int)t);
    return false;
  }
  const float* base = p.cos_sin + pair0;
  auto pick = [&](uint32_t axis) {
    const int r = axis == 0 ? row[0] : axis == 1 ? row[1] : axis == 2 ? row[2] : row[3];
    return base + (int64_t)r * p.rot;
  };
  const uint32_t ax = axes == 1 ? 0u : p.pair_axis[pair0 >> 4] >> (2 * (pair0 & 15));   // 8 (4) pairs
  float c[8], s[8];
  const int n = p.adjacent ? 1 : 2;   // quads of pairs
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h >= n) break;
    if (axes == 1 || p.quads) {
      const float* src = pick((ax >> (8 * h)) & 3u) + 4 * h;
      const float4 x = __ldg(reinterpret_cast<const float4*>(src));
      const float4 y = __ldg(reinterpret_cast<const float4*>(src + half));
      c[4 * h] = x.x, c[4 * h + 1] = x.y, c[4 * h + 2] = x.z, c[4 * h + 3] = x.w;
      s[4 * h] = y.x, s[4 * h + 1] = y.y, s[4 * h + 2] = y.z, s[4 * h + 3] = y.w;
    } else {
#pragma unroll
      for (int e = 4 * h; e < 4 * h + 4; ++e) {
        const float* src = pick((ax >> (2 * e)) & 3u) + e;
        c[e] = __ldg(src);
        s[e] = __ldg(src + half);
      }
    }
  }
  if (p.adjacent) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a.c[e] = make_float2(c[e], c[e]);
      a.s[e] = make_float2(-s[e], s[e]);
    }
  } else {
    const bool lower = 8 * o < half;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a.c[e] = make_float2(c[2 * e], c[2 * e + 1]);
      a.s[e] = make_float2(lower ? -s[2 * e] : s[2 * e], lower ? -s[2 * e + 1] : s[2 * e + 1]);
    }
  }
  return true;
}

// The rotated values of a lane's 8 dims x (bf16), y the other dims of their pairs.  The
// products are multiply-adds of p.neg_zero, -0: mul.rn.f32x2 and add.rn.f32x2 came out fused
// now and then, results a last place off.
__device__ __forceinline__ void turn8(const RopeParams& p, const uint4& x, const uint4& y, const Turn& a, float2 (&f)[4]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
  const float2 nz = make_float2(p.neg_zero, p.neg_zero);
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = add2(fma2(bf16_2(w[k]), a.c[k], nz), fma2(bf16_2(v[k]), a.s[k], nz));
}

__device__ __forceinline__ void plain8(const uint4& x, float2 (&f)[4]) {
  f[0] = bf16_2(x.x), f[1] = bf16_2(x.y), f[2] = bf16_2(x.z), f[3] = bf16_2(x.w);
}

__device__ __forceinline__ uint4 shfl4(const uint4& x, int lane) {
  return make_uint4(__shfl_sync(0xffffffffu, x.x, lane), __shfl_sync(0xffffffffu, x.y, lane),
                    __shfl_sync(0xffffffffu, x.z, lane), __shfl_sync(0xffffffffu, x.w, lane));
}

// The other dims of the pairs of a lane's 8: its own, neighbours swapped, or lane `from`'s.
__device__ __forceinline__ uint4 partners(const RopeParams& p, const uint4& x, int from) {
  if (p.adjacent)
    return make_uint4(__byte_perm(x.x, 0, 0x1032), __byte_perm(x.y, 0, 0x1032), __byte_perm(x.z, 0, 0x1032),
                      __byte_perm(x.w, 0, 0x1032));
  return shfl4(x, from);
}

__device__ __forceinline__ uint4 bf16x8_of(const float2 (&f)[4]) {
  return make_uint4(bf16x2_of(f[0].x, f[0].y), bf16x2_of(f[1].x, f[1].y), bf16x2_of(f[2].x, f[2].y),
                    bf16x2_of(f[3].x, f[3].y));
}

template <int KV>
constexpr bool is_four() { return KV == PA_KV_INT4 || KV == PA_KV_FP4_E2M1; }

// Four quotients -> their 8-bit codes, the first in the lowest byte (int8: not NaN).
template <int KV>
__device__ __forceinline__ uint32_t codes4(const float* v) {
  if constexpr (KV == PA_KV_FP8_E4M3) {
    uint32_t w;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
    return w;
  } else {
    // adding 2^23 + 2^22 rounds to an integer, ties to even, and leaves it in the low bits
    uint32_t t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = __float_as_uint(fminf(fmaxf(v[k], -127.0f), 127.0f) + 12582912.0f);
    return __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// max |x|, NaN if there is one
__device__ __forceinline__ float max_abs8(const float2 (&x)[4]) {
  return max3_abs_nan(max3_abs_nan(x[0].x, x[0].y, x[1].x), max3_abs_nan(x[1].y, x[2].x, x[2].y),
                      max3_abs_nan(x[3].x, x[3].y, 0.0f));
}

// Whether quot() gives the quotients of values below 2^60 by s.
__device__ __forceinline__ bool short_by(float s) { return s > 0x1p-60f && s < 0x1p60f; }

// Any quotient, as pa_cache.cu's writer takes it (a NaN counts as 0 for int8).
template <int KV>
__device__ __forceinline__ float any_quotient(float x, float s) {
  const float v = __fdiv_rn(x, s);
  return KV == PA_KV_INT8 && v != v ? 0.0f : v;
}

// The quotients that codes4 takes where short_by holds.  E4M3 keeps a zero's sign and quot2 makes
// every zero +0, so there it is -x / d by the same steps, whose zeros' signs are turned too, and
// `kTurn` turns the codes' signs back.
template <int KV>
constexpr uint32_t kTurn = KV == PA_KV_FP8_E4M3 ? 0x80808080u : 0u;

template <int KV>
__device__ __forceinline__ float2 short_quotients(float2 x, float2 d, float2 r) {
  if constexpr (KV == PA_KV_FP8_E4M3) {
    const float2 nr = make_float2(-r.x, -r.y), n = mul2(x, nr);
    return fma2(fma2(n, d, x), nr, n);
  } else {
    return quot2(x, d, r);
  }
}

// Eight values over their scales (r = 1 / s; ok: short_by of the scales) -> two words of
// 8-bit codes.
template <int KV, bool PC>
__device__ __forceinline__ uint2 codes8_of(const float2 (&x)[4], const float2* s, const float2* r, bool ok) {
  float2 v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = short_quotients<KV>(x[e], s[PC ? e : 0], r[PC ? e : 0]);
  uint32_t turn = kTurn<KV>;
  if (!(max_abs8(x) < 0x1p60f) || !ok) {
    turn = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 d = s[PC ? e : 0];
      v[e] = make_float2(any_quotient<KV>(x[e].x, d.x), any_quotient<KV>(x[e].y, d.y));
    }
  }
  return make_uint2(codes4<KV>(&v[0].x) ^ turn, codes4<KV>(&v[2].x) ^ turn);
}

// A K row's 8 values of a lane, 4 bits, by divisions: codes and the block's scale.
template <int FP4, bool PC>
__device__ __forceinline__ void any_k4(const float2 (&f)[4], const float2* g, uint8_t* slab, int off, int c, bool in) {
  constexpr float kTop = Fmt<FP4>::kTop;
  float x[8], a = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = e & 1 ? f[e >> 1].y : f[e >> 1].x;
    if (x[e] != x[e]) x[e] = 0.0f;
    a = fmaxf(a, fabsf(__fdiv_rn(x[e], PC && (e & 1) ? g[e >> 1].y : g[PC ? e >> 1 : 0].x)));
  }
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  const uint32_t sb = block_scale<FP4>(__fdiv_rn(a, kTop));
  const float t = e4m3_to_f32(sb);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float step = __fmul_rn(t, PC && (e & 1) ? g[e >> 1].y : g[PC ? e >> 1 : 0].x);
    x[e] = fminf(fmaxf(step > 0.0f ? __fdiv_rn(x[e], step) : 0.0f, -kTop), kTop);
  }
  const uint32_t w = pack8<FP4>(x);
  if (in) {
    *reinterpret_cast<uint32_t*>(slab + k4_code_off(off, 8 * c)) = w;
    if ((c & 1) == 0) slab[k4_scale_off(off, c >> 1)] = (uint8_t)sb;
  }
}

template <int FP4>
__device__ __forceinline__ uint32_t pack4x2(const float2 (&q)[4]) {
  const float v[8] = {q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
  return pack8<FP4>(v);
}

// A lane's 8 values of a K row -> its codes (and block scale), in place within the slab.
// The lanes of a block are neighbours; every lane of the warp calls it, those of rows
// outside the range with in = false.  (4 bits: per-channel scales, store_k4 has the others.)
template <int KV, bool PC>
__device__ __forceinline__ void store_k(const RopeParams& p, const float2 (&f)[4], uint8_t* slab, int kvh, int off, int c,
                                        bool in) {
  float2 g[4], rg[4];
  bool ok = true;
  if constexpr (PC) {
    const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(p.a.k_scale) + kvh * kV4Dim + 8 * c;
    if (p.k_scale16) {
      plain8(__ldg(reinterpret_cast<const uint4*>(sc)), g);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = make_float2(__bfloat162float(sc[2 * e]), __bfloat162float(sc[2 * e + 1]));
    }
  } else {
    g[0].x = g[0].y = load_scale(p.a.k_scale, p.a.scale_kind, kvh);
  }
#pragma unroll
  for (int e = 0; e < (PC ? 4 : 1); ++e) {
    rg[e].x = rcp_approx(g[e].x);
    rg[e].y = PC ? rcp_approx(g[e].y) : rg[e].x;
    ok = ok && short_by(g[e].x) && short_by(g[e].y);
  }
  if constexpr (!is_four<KV>()) {
    const uint2 w = codes8_of<KV, PC>(f, g, rg, ok);
    if (in) *reinterpret_cast<uint2*>(slab + off * kV4Dim + 8 * c) = w;
  } else {
    constexpr int FP4 = KV == PA_KV_FP4_E2M1;
    constexpr float kTop = Fmt<FP4>::kTop;
    // the block's maximum of |x / g| by short quotients; a NaN, or a block out of their
    // range, shows in `fine`
    float2 q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = quot2(f[e], g[e], rg[e]);
    float a = max_abs8(q);
    a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 1));
    const uint32_t sb = block_scale<FP4>(quot(a, kTop, 1.0f / kTop));
    const float s = e4m3_to_f32(sb), rs = rcp_approx(s);
    const float2 s2 = make_float2(s, s), rs2 = make_float2(rs, rs);
    float low = 1e30f, high = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 st = mul2(s2, g[e]);
      low = fminf(low, fminf(fabsf(st.x), fabsf(st.y)));
      high = fmaxf(high, fmaxf(fabsf(st.x), fabsf(st.y)));
      q[e] = quot2(f[e], st, mul2(rs2, rg[e]));
    }
    const bool fine = ok && common<FP4>(a, s, low) && high < 1e30f;
    if (__all_sync(0xffffffffu, fine || !in)) {
      const uint32_t w = pack4x2<FP4>(q);
      if (in) {
        *reinterpret_cast<uint32_t*>(slab + k4_code_off(off, 8 * c)) = w;
        if ((c & 1) == 0) slab[k4_scale_off(off, c >> 1)] = (uint8_t)sb;
      }
    } else {
      any_k4<FP4, true>(f, g, slab, off, c, in);
    }
  }
}

// The K rows of two neighbouring heads, kvh and kvh + 1, 4 bits, a scale a head or for all:
// a lane of a block works out the scale of one of them.  `slab` is head kvh's; in0, in1:
// whether the row is to be written (kvh may be -1, or the last head, with the other's false).
template <int KV>
__device__ __forceinline__ void store_k4(const RopeParams& p, const float2 (&f)[2][4], uint8_t* slab, int kvh, int off, int c,
                                         bool in0, bool in1) {
  constexpr int FP4 = KV == PA_KV_FP4_E2M1;
  constexpr float kTop = Fmt<FP4>::kTop;
  const bool odd = c & 1;
  const int mine = kvh + (odd ? 1 : 0);
  const float g = load_scale(p.a.k_scale, p.a.scale_kind, min(max(mine, 0), p.a.kv_heads - 1));
  const float a0 = max_abs8(f[0]), a1 = max_abs8(f[1]);
  const float m = max_nan(odd ? a1 : a0, __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1));
  // of the largest: rounding keeps the order
  const float a = fabsf(quot(m, g, rcp_approx(g)));
  const uint32_t sb = block_scale<FP4>(quot(a, kTop, 1.0f / kTop));
  const float s = e4m3_to_f32(sb), st = s * g, rs = rcp_approx(st);
  const bool in = odd ? in1 : in0, fine = short_by(g) && common<FP4>(a, s, fabsf(st));
  uint8_t* codes = slab + k4_code_off(off, 8 * c);
  if (__all_sync(0xffffffffu, fine || !in)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int from = (threadIdx.x & 30) | i;
      const float si = __shfl_sync(0xffffffffu, st, from), ri = __shfl_sync(0xffffffffu, rs, from);
      const float2 s2 = make_float2(si, si), r2 = make_float2(ri, ri);
      float2 q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = quot2(f[i][e], s2, r2);
      const uint32_t w = pack4x2<FP4>(q);
      if (i ? in1 : in0) *reinterpret_cast<uint32_t*>(codes + i * kV4Slab) = w;
    }
    if (in) slab[(odd ? kV4Slab : 0) + k4_scale_off(off, c >> 1)] = (uint8_t)sb;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float gi = __shfl_sync(0xffffffffu, g, (threadIdx.x & 30) | i);
      const float2 g2[1] = {make_float2(gi, gi)};
      any_k4<FP4, false>(f[i], g2, slab + i * kV4Slab, off, c, i ? in1 : in0);
    }
  }
}

// V of an 8-bit cache: the unit's positions [a, e) of U (FULL: all), lane = 4 dims.
template <int KV, bool PC, int U, bool FULL>
__device__ __forceinline__ void store_v8(const RopeParams& p, const __nv_bfloat16* rows, uint8_t* slab, int kvh, int off0,
                                         int a, int e, int lane) {
  float2 g[2], rg[2];
#pragma unroll
  for (int d = 0; d < (PC ? 2 : 1); ++d) {
    g[d].x = load_scale(p.a.v_scale, p.a.scale_kind, PC ? kvh * kV4Dim + 4 * lane + 2 * d : kvh);
    g[d].y = PC ? load_scale(p.a.v_scale, p.a.scale_kind, kvh * kV4Dim + 4 * lane + 2 * d + 1) : g[d].x;
  }
  bool ok = true;
#pragma unroll
  for (int d = 0; d < (PC ? 2 : 1); ++d) {
    rg[d] = make_float2(rcp_approx(g[d].x), rcp_approx(g[d].y));
    ok = ok && short_by(g[d].x) && short_by(g[d].y);
  }
  const __nv_bfloat16* src = rows + 4 * lane - (FULL ? 0 : (int64_t)a * p.a.kv_stride);
  uint8_t* dst = slab + 4 * lane * kPage + off0;
  uint32_t w[4][U / 4];
#pragma unroll
  for (int k = 0; k < U; k += 8) {
    uint2 x[8];
    uint32_t top = 0;   // the largest exponents and mantissas
#pragma unroll
    for (int j = 0; j < 8; ++j, src += p.a.kv_stride) {
      x[j] = FULL || (k + j >= a && k + j < e) ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
      top = max_u16x2(top, max_u16x2(x[j].x & 0x7FFF7FFFu, x[j].y & 0x7FFF7FFFu));
    }
    // all below 2^60 (bf16 0x5D80)
    const bool fine = ok && (top & 0xFFFFu) < 0x5D80u && (top >> 16) < 0x5D80u;
#pragma unroll
    for (int d = 0; d < 4; d += 2) {
      const float2 gd = g[PC ? d / 2 : 0], rd = rg[PC ? d / 2 : 0];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v0[4], v1[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = short_quotients<KV>(bf16_2(d ? x[4 * h + j].y : x[4 * h + j].x), gd, rd);
          v0[j] = v.x;
          v1[j] = v.y;
        }
        if (!fine) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = bf16_2(d ? x[4 * h + j].y : x[4 * h + j].x);
            v0[j] = any_quotient<KV>(f.x, gd.x);
            v1[j] = any_quotient<KV>(f.y, gd.y);
          }
        }
        w[d][k / 4 + h] = codes4<KV>(v0) ^ (fine ? kTurn<KV> : 0);
        w[d + 1][k / 4 + h] = codes4<KV>(v1) ^ (fine ? kTurn<KV> : 0);
      }
    }
  }
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint8_t* to = dst + d * kPage;
    if constexpr (FULL && U == 32) {   // whole sectors
      if (p.v32) {
        st_global_32(to, w[d]);
      } else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(w[d][0], w[d][1], w[d][2], w[d][3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(w[d][4], w[d][5], w[d][6], w[d][7]);
      }
    } else if constexpr (FULL) {
#pragma unroll
      for (int k = 0; k < U; k += 8) *reinterpret_cast<uint2*>(to + k) = make_uint2(w[d][k / 4], w[d][k / 4 + 1]);
    } else {   // only the range's own positions
#pragma unroll
      for (int k = 0; k < U; k += 8) {
        if (a <= k && k + 8 <= e) {
          *reinterpret_cast<uint2*>(to + k) = make_uint2(w[d][k / 4], w[d][k / 4 + 1]);
        } else {
#pragma unroll
          for (int j = k; j < k + 8; ++j)
            if (j >= a && j < e) to[j] = (uint8_t)(w[d][j >> 2] >> (8 * (j & 3)));
        }
      }
    }
  }
}

// The page of position `pos` of sequence b, or -1 (and the status recorded).
__device__ __forceinline__ int page_at(const RopeParams& p, int b, int pos, int lane) {
  const int lp = pos / kPage;
  const int page = lp < p.a.max_blocks ? p.a.block_table[(int64_t)b * p.a.max_blocks + lp] : -1;
  if (page >= 0 && page < p.a.num_pages) return page;
  if (lane == 0) record_status(p.a.status, PA_ERR_BAD_PAGE, b);
  return -1;
}

// A unit of positions: sequence, first position, and the range's part [lo, hi) of it.
struct UnitAt {
  int b, u0, lo, hi;
  int64_t row;   // token row of position lo
};

__device__ __forceinline__ bool unit_at(const RopeParams& p, int shift, const RowUnits& units, uint32_t n, int lane,
                                        UnitAt& m) {
  int u;
  find_unit_of(shift, units, p.a.cu_seqlens_q, n, lane, m.b, u);
  const int q = p.a.seq_lens[m.b];
  if (q <= 0) return false;
  const int start = p.a.seq_lens_kv[m.b], end = start + q;
  m.u0 = ((start >> shift) + u) << shift;
  m.lo = max(m.u0, start);
  m.hi = min(m.u0 + (1 << shift), end);
  m.row = (int64_t)p.a.cu_seqlens_q[m.b] + (m.lo - start);
  return m.lo < m.hi;
}

// ---- GQA
// Queries alone, of many rows: few registers, so that 32 warps an SM have their loads on
// the way (in one kernel with K's and V's quantisers 16; 35k rows of 32 heads 128 us)
__global__ void __launch_bounds__(kWarps * 32, kQCtas) rope_q_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31;
  const uint32_t id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= p.rot_warps) return;
  const uint32_t bu = id / (uint32_t)p.groups;
  const int g0 = (int)(id - bu * p.groups) * p.group_heads, g1 = min(p.q_heads, g0 + p.group_heads);
  UnitAt m;
  if (!unit_at(p, p.unit_shift, p.units, bu, lane, m)) return;
  const int c = lane & 15, oct = p.rot / 8;
  const bool turned = c < oct;
  const int other = !turned ? lane : (lane & 16) | (c < oct / 2 ? c + oct / 2 : c - oct / 2);
  for (int r = m.lo; r < m.hi; r += 2) {
    const int pos = r + (lane >> 4);
    const bool in = pos < m.hi;
    const int64_t t = m.row + (pos - m.lo);
    const __nv_bfloat16* src = p.q + t * p.q_stride + 8 * c;
    __nv_bfloat16* dst = p.q_out + t * p.q_out_stride + 8 * c;
    uint4 x[4];
    auto load = [&](int h0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] = make_uint4(0, 0, 0, 0);
        if (in && h0 + k < g1) x[k] = *reinterpret_cast<const uint4*>(src + (h0 + k) * kV4Dim);
      }
    };
    load(g0);
    Turn a;
    const bool turn = in && turned && load_turn(p, t, pos, c, a);
    for (int h0 = g0; h0 < g1; h0 += 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (h0 + k >= g1) break;
        const uint4 y = partners(p, x[k], other);
        float2 f[4];
        if (turn) turn8(p, x[k], y, a, f);
        else plain8(x[k], f);
        if (in) *reinterpret_cast<uint4*>(dst + (h0 + k) * kV4Dim) = bf16x8_of(f);
      }
      if (h0 + 4 < g1) load(h0 + 4);
    }
  }
}

// Everything in one launch (U = 8, few rows), or K and V (U = 32; 35k rows of 8 heads: FP4
// 58 us, int4 61, int8 67, E4M3 63, their bytes 27 and 33; per-channel scales 88, 99, 80 and 78,
// 5 less than with 32 warps an SM, which spill more; on three axes 4 to 6 more).  K alone takes
// 45 and V 23 (FP4): instructions (47 % of the issue slots at 32 % of the warps) and loads in
// turn; the next heads' rows requested ahead 62 to 70, 4 heads at once 60 to 68.  4-bit blocks
// below E4M3's normal range go by divisions, and with one of them all of a K step or V unit: the
// same rows on three axes times 0.03 with scales of 1 353 us (FP4; int4 356) of 63 (65), every
// 16th row 0 338 (340).
template <int KV, bool PC, int U>
__global__ void __launch_bounds__(kWarps * 32, U == 8 ? 2 : PC ? 3 : 4) rope_append_kernel(const RopeParams p) {
  constexpr int kBatch = U == 8 ? 4 : 2;   // heads whose rows are on the way at once
  const int lane = threadIdx.x & 31;
  const uint32_t id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  constexpr int kSlabBytes = is_four<KV>() ? kV4Slab : kPage * kV4Dim;
  UnitAt m;
  if (id >= p.rot_warps) {   // V
    const uint32_t n = id - p.rot_warps;
    if (n >= p.a.total) return;
    const uint32_t bu = n / (uint32_t)p.a.kv_heads;
    const int kvh = (int)(n - bu * p.a.kv_heads);
    if (!unit_at(p, U == 8 ? 3 : 5, p.a.units, bu, lane, m)) return;
    const int page = page_at(p, m.b, m.u0, lane);
    if (page < 0) return;
    const __nv_bfloat16* rows = p.a.v_new + m.row * p.a.kv_stride + (int64_t)kvh * kV4Dim;
    uint8_t* slab = p.a.cache_v + ((int64_t)page * p.a.kv_heads + kvh) * kSlabBytes;
    const int a = m.lo - m.u0, e = m.hi - m.u0;
    if constexpr (is_four<KV>()) {
      constexpr int FP4 = KV == PA_KV_FP4_E2M1;
      uint8_t* half = slab + m.u0 % kPage / kV4Half * kV4HalfBytes;
      const int first = m.u0 % kV4Half;
      e - a == U ? write_v<FP4, PC, U, true>(p.a, rows, half, kvh, first, a, e, lane)
                 : write_v<FP4, PC, U, false>(p.a, rows, half, kvh, first, a, e, lane);
    } else {
      e - a == U ? store_v8<KV, PC, U, true>(p, rows, slab, kvh, m.u0 % kPage, a, e, lane)
                 : store_v8<KV, PC, U, false>(p, rows, slab, kvh, m.u0 % kPage, a, e, lane);
    }
    return;
  }
  // rotation: head group fastest, so that neighbouring warps read the same rows
  const uint32_t bu = id / (uint32_t)p.groups;
  const int g0 = (int)(id - bu * p.groups) * p.group_heads;
  const int heads = p.q_heads + p.a.kv_heads, g1 = min(heads, g0 + p.group_heads);
  if (!unit_at(p, p.unit_shift, p.units, bu, lane, m)) return;
  const int page = g1 > p.q_heads ? page_at(p, m.b, m.u0, lane) : -1;
  const int c = lane & 15, oct = p.rot / 8;
  const bool turned = c < oct;
  // the lane whose dims are the other halves of this one's pairs
  const int other = !turned ? lane : (lane & 16) | (c < oct / 2 ? c + oct / 2 : c - oct / 2);
  for (int r = m.lo; r < m.hi; r += 2) {
    const int pos = r + (lane >> 4);
    const bool in = pos < m.hi;
    const int64_t t = m.row + (pos - m.lo);
    Turn a;
    const bool turn = in && turned && load_turn(p, t, pos, c, a);
    const __nv_bfloat16* q_row = p.q + t * p.q_stride + 8 * c;
    const __nv_bfloat16* k_row = p.a.k_new + t * p.a.kv_stride - p.q_heads * kV4Dim + 8 * c;   // of head h: + h * 128
    __nv_bfloat16* q_to = p.q_out + t * p.q_out_stride + 8 * c;
    uint8_t* slabs = p.a.cache_k + (int64_t)page * p.a.kv_heads * kSlabBytes;
    for (int h0 = g0; h0 < g1; h0 += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int h = h0 + k;
        x[k] = make_uint4(0, 0, 0, 0);
        if (in && h < g1) x[k] = *reinterpret_cast<const uint4*>((h < p.q_heads ? q_row : k_row) + h * kV4Dim);
      }
      // the rotated values of head h0 + k; a query's are written
      auto rotate = [&](int k, float2 (&f)[4]) {
        const uint4 y = partners(p, x[k], other);
        if (turn) turn8(p, x[k], y, a, f);
        else plain8(x[k], f);
        if (in && h0 + k < min(g1, p.q_heads)) *reinterpret_cast<uint4*>(q_to + (h0 + k) * kV4Dim) = bf16x8_of(f);
      };
      constexpr int kStep = is_four<KV>() && !PC ? 2 : 1;
#pragma unroll
      for (int k = 0; k < kBatch; k += kStep) {
        const int h = h0 + k, kvh = h - p.q_heads;
        if (h >= g1) break;
        uint8_t* slab = slabs + (int64_t)kvh * kSlabBytes;
        if constexpr (kStep == 2) {
          float2 f[2][4];
          rotate(k, f[0]);
          rotate(k + 1, f[1]);
          if (page >= 0 && kvh + 1 >= 0) store_k4<KV>(p, f, slab, kvh, pos % kPage, c, in && kvh >= 0, in && h + 1 < g1);
        } else {
          float2 f[4];
          rotate(k, f);
          if (page >= 0 && kvh >= 0) store_k<KV, PC>(p, f, slab, kvh, pos % kPage, c, in);
        }
      }
    }
  }
}

// ---- MLA: groups of query heads, and one more for the latent row
template <int KV>
__global__ void __launch_bounds__(kWarps * 32, 3) rope_latent_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31;
  const uint32_t id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= p.rot_warps) return;
  const uint32_t bu = id / (uint32_t)p.groups;
  const int g0 = (int)(id - bu * p.groups) * p.group_heads;
  UnitAt m;
  if (!unit_at(p, p.unit_shift, p.units, bu, lane, m)) return;
  const int o = lane & 7, oct = p.rot / 8;
  const bool turned = o < oct;
  const int other = !turned ? lane : (lane & 24) | (o < oct / 2 ? o + oct / 2 : o - oct / 2);
  if (g0 >= p.q_heads) {   // the rows of the cache
    const int page = page_at(p, m.b, m.u0, lane);
    if (page < 0) return;
    const float scale = load_scale(p.a.k_scale, PA_SCALE_GLOBAL, 0), rcp = rcp_approx(scale);
    const float2 s[1] = {make_float2(scale, scale)}, rs[1] = {make_float2(rcp, rcp)};
    for (int pos = m.lo; pos < m.hi; ++pos) {
      const int64_t t = m.row + (pos - m.lo);
      const __nv_bfloat16* src = p.a.k_new + t * p.a.kv_stride;
      uint8_t* dst = p.a.cache_k + ((int64_t)page * kPage + pos % kPage) * kMlaRow;
      uint4 x[3] = {};
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k < 2 || lane < 8) x[k] = *reinterpret_cast<const uint4*>(src + 8 * (lane + 32 * k));
      Turn a;
      const bool turn = lane < 8 && turned && load_turn(p, t, pos, o, a);
      const uint4 y = partners(p, x[2], other);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (k == 2 && lane >= 8) break;
        float2 f[4];
        if (k == 2 && turn) turn8(p, x[2], y, a, f);
        else plain8(x[k], f);
        *reinterpret_cast<uint2*>(dst + 8 * (lane + 32 * k)) = codes8_of<KV, false>(f, s, rs, short_by(scale));
      }
    }
    return;
  }
  const bool copy = p.q_out != p.q;   // dims before the rotated ones; they stay in place
  const int g1 = min(p.q_heads, g0 + p.group_heads);
  for (int pos = m.lo; pos < m.hi; ++pos) {
    const int64_t t = m.row + (pos - m.lo);
    const __nv_bfloat16* src = p.q + t * p.q_stride;
    __nv_bfloat16* dst = p.q_out + t * p.q_out_stride;
    Turn a;
    const bool turn = turned && load_turn(p, t, pos, o, a);
    const int at = (lane >> 3) * kMlaQ + kMlaNope + 8 * o, at0 = (lane >> 4) * kMlaQ + 8 * (lane & 15);
    for (int h0 = g0; h0 < g1; h0 += 8) {   // the heads are a multiple of eight
      uint4 x[2], n[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) x[k] = *reinterpret_cast<const uint4*>(src + (h0 + 4 * k) * kMlaQ + at);
      if (copy) {
#pragma unroll
        for (int k = 0; k < 4; ++k) n[k] = *reinterpret_cast<const uint4*>(src + (h0 + 2 * k) * kMlaQ + at0);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 y = partners(p, x[k], other);
        float2 f[4];
        if (turn) turn8(p, x[k], y, a, f);
        else plain8(x[k], f);
        *reinterpret_cast<uint4*>(dst + (h0 + 4 * k) * kMlaQ + at) = bf16x8_of(f);
      }
      if (copy) {
#pragma unroll
        for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(dst + (h0 + 2 * k) * kMlaQ + at0) = n[k];
      }
    }
  }
}

template <int KV, int U>
cudaError_t launch_gqa(RopeParams& p, const Plan& plan, cudaStream_t stream) {
  p.a.units = row_units<U>(plan.prob.bsz, plan.max_q, plan.total_q);
  const double v = (double)p.a.units.count * plan.prob.kv_heads;
  if (v + p.rot_warps > (double)INT32_MAX) return cudaErrorInvalidValue;
  p.a.total = (uint32_t)v;
  const dim3 grid((p.rot_warps + p.a.total + kWarps - 1) / kWarps), block(kWarps * 32);
  if (p.a.scale_kind == PA_SCALE_PER_CHANNEL) rope_append_kernel<KV, true, U><<<grid, block, 0, stream>>>(p);
  else rope_append_kernel<KV, false, U><<<grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int KV>
cudaError_t launch_kv(RopeParams& p, const Plan& plan, bool small, cudaStream_t stream) {
  return small ? launch_gqa<KV, 8>(p, plan, stream) : launch_gqa<KV, 32>(p, plan, stream);
}

}  // namespace

cudaError_t launch_rope_append(const Plan& plan, const pa_args& a, const pa_rope& rope, const void* q,
                               int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k_new,
                               const void* v_new, int64_t kv_stride, int32_t* status, cudaStream_t stream) {
  const pa_problem& pr = plan.prob;
  if (pr.bsz == 0 || plan.max_q == 0) return cudaSuccess;
  RopeParams p{};
  p.a.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.a.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.a.kv_stride = kv_stride;
  p.a.cache_k = static_cast<uint8_t*>(const_cast<void*>(a.cache_k));
  p.a.cache_v = static_cast<uint8_t*>(const_cast<void*>(a.cache_v));
  p.a.k_scale = a.k_scale;
  p.a.v_scale = a.v_scale;
  p.a.block_table = a.block_table;
  p.a.seq_lens = a.seq_lens;
  p.a.seq_lens_kv = a.seq_lens_kv;
  p.a.cu_seqlens_q = a.cu_seqlens_q;
  p.a.status = status;
  p.a.max_blocks = pr.max_blocks_per_seq;
  p.a.num_pages = pr.num_pages;
  p.a.kv_heads = pr.kv_heads;
  p.a.scale_kind = pr.scale_kind;
  p.a.vec = 1;
  p.k_scale16 = reinterpret_cast<uintptr_t>(a.k_scale) % 16 == 0;
  p.v32 = reinterpret_cast<uintptr_t>(a.cache_v) % 32 == 0;
  p.cos_sin = rope.cos_sin;
  p.positions = rope.positions;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_stride = q_stride;
  p.q_out_stride = q_out_stride;
  p.q_heads = q ? pr.q_heads : 0;
  p.table_rows = rope.table_rows;
  p.rot = rope.rot_dim;
  p.adjacent = rope.pairs == PA_ROPE_ADJACENT;
  p.axes = rope.axes;
  p.total_q = plan.total_q;
  p.neg_zero = -0.0f;
  p.quads = 1;
  for (int i = 0; i < rope.rot_dim / 2; ++i) {
    p.pair_axis[i >> 4] |= (uint32_t)(rope.pair_axis[i] & 3) << (2 * (i & 15));
    if (rope.pair_axis[i] != rope.pair_axis[i & ~3]) p.quads = 0;
  }
  const bool mla = pr.layout == PA_LAYOUT_MLA;
  // One launch for all while rows are few, V by units of 8; then the queries by themselves
  // and V by units of 32.  Rows of all heads an SM, us in one launch and in two, FP4: 2048
  // rows of 40 heads 20.7 and 20.4, 1024 12.7 and 18.7, 4096 35.6 and 29.0; 4096 rows of 18
  // 17.6 and 20.3, 6144 23.0 and 21.5; without queries, where both are one launch, 2048
  // rows of 8 heads 10.6 and 10.6, 1024 8.2 and 10.4, 4096 14.7 and 12.7.
  const bool small = (double)plan.total_q * (p.q_heads + pr.kv_heads) < (q ? 560.0 : 150.0) * plan.num_sms;
  // Positions of a rotation warp's unit: a warp has all heads of a row, or 8 to 16, and reads
  // its cos and sin once; with many rows 8, so that what a unit begins with is shared, with
  // fewer 4 or 2, so that there are 16 units an SM.  Units of 2, 4 and 8, us (40 heads, FP4):
  // 6144 rows 39, 44, 56, 12800 66, 66, 78, 16384 84, 82, 88, 35200 157, 155, 153.  (K and V of
  // 35k rows by units of 8 and 2 of 8 heads, to have as many warps, 94 us, all heads 60; K's
  // warps among V's instead of before them 76: theirs are the long ones.)
  p.unit_shift = 1;
  if (!mla && !small)
    while (p.unit_shift < 3 && plan.total_q >= (16 << (p.unit_shift + 1)) * (int64_t)plan.num_sms) ++p.unit_shift;
  p.units = row_units_of(1 << p.unit_shift, pr.bsz, plan.max_q, plan.total_q);
  // Heads of a warp: enough to use a row's cos and sin often, few while the warps would
  // not fill the GPU
  auto share = [&](int heads, int least, int most = 16) {
    p.group_heads = most;
    while (p.group_heads > least &&
           (double)p.units.count * ((heads + p.group_heads - 1) / p.group_heads) < 16.0 * kWarps * plan.num_sms)
      p.group_heads /= 2;
    p.groups = (heads + p.group_heads - 1) / p.group_heads + (mla ? 1 : 0);
    const double rot = (double)p.units.count * p.groups;
    p.rot_warps = rot > (double)INT32_MAX ? 0 : (uint32_t)rot;
    return p.rot_warps > 0;
  };
  if (!mla && q && !small) {
    // 8 or 16 heads, by the time of the waves of warps (24k rows of 32 heads: 16 in 1.24 waves
    // 59 us, 8 in 2.47 50; 35k: 16 in 1.81 waves 94, 8 in 3.63 98)
    auto waves = [&](int g) {
      const double warps = ((double)plan.total_q / (1 << p.unit_shift) + pr.bsz) * ((p.q_heads + g - 1) / g);   // that have rows
      return std::ceil(warps / (kQCtas * kWarps * plan.num_sms)) * (std::min(g, p.q_heads) + 2);
    };
    const int g = waves(8) < waves(16) ? 8 : 16;
    if (!share(p.q_heads, g, g)) return cudaErrorInvalidValue;
    rope_q_kernel<<<(p.rot_warps + kWarps - 1) / kWarps, kWarps * 32, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.q_heads = 0;
  }
  if (!share(p.q_heads + (mla ? 0 : pr.kv_heads), mla || !small ? 8 : 4)) return cudaErrorInvalidValue;
  if (mla) {
    const dim3 grid((p.rot_warps + kWarps - 1) / kWarps), block(kWarps * 32);
    if (pr.kv_dtype == PA_KV_FP8_E4M3) rope_latent_kernel<PA_KV_FP8_E4M3><<<grid, block, 0, stream>>>(p);
    else rope_latent_kernel<PA_KV_INT8><<<grid, block, 0, stream>>>(p);
    return cudaGetLastError();
  }
  switch (pr.kv_dtype) {
    case PA_KV_INT8: return launch_kv<PA_KV_INT8>(p, plan, small, stream);
    case PA_KV_FP8_E4M3: return launch_kv<PA_KV_FP8_E4M3>(p, plan, small, stream);
    case PA_KV_INT4: return launch_kv<PA_KV_INT4>(p, plan, small, stream);
    default: return launch_kv<PA_KV_FP4_E2M1>(p, plan, small, stream);
  }
}

}  // namespace pa
