// pa_cache4.cu - quantise-and-write of the appended tokens' K / V into the
// 4-bit paged cache.
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
// One warp per (sequence, half page of the appended range, kv head, K or V),
// each reading its rows once with coalesced 8- or 16-byte loads:
//   K: lane = 8 dims of one row (two lanes per block), codes leave as a 32-bit
//      word per lane;
//   V: lane = 4 dims of all 32 positions (four lanes per block), so a dim's 16
//      code bytes of the half page gather in the lane's registers and leave as
//      one store; a half page that is written in part keeps the other nibbles
//      (one warp owns a half page, so nobody else writes its bytes).
// The block maximum of uniform scales is taken on the bf16 bits, two elements a
// step; the lanes of a block then work out a different row's scale each and
// share them.  Quotients: an approximate reciprocal, and one correction of the
// quotient by its residual, which gives every quotient that is exactly a border
// between two codes exactly, and the others to the last bit; blocks out of the
// common range (a scale that is not a normal E4M3 number, saturated, infinities,
// NaN) take the division.
// What bounds it: 2.56 bytes per element against about 8 instructions.
#include "pa_common.cuh"
#include "pa_kv4.cuh"

namespace pa {
namespace {

constexpr int kPage = 64;
constexpr int kWarps = 8;

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
  int32_t units;       // half pages an appended range can touch
  int32_t vec;         // rows may be read with 16-byte loads
  uint32_t total;      // (sequence, half page, kv head, side) warps
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

// x / d with r close to 1 / d: the quotient corrected once by its residual
__device__ __forceinline__ float quot(float x, float d, float r) {
  const float q = x * r;
  return __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int FP4>
struct Fmt {
  static constexpr float kTop = FP4 ? 6.0f : 7.0f;
};

// Block scale from a = max |x / g|: the E4M3 byte.
template <int FP4>
__device__ __forceinline__ uint32_t block_scale(float a) {
  uint16_t sb;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.0f), "f"(__fdiv_rn(a, Fmt<FP4>::kTop)));
  return sb & 0xFFu;
}

// Whether the short quotients hold for a block: a normal, unsaturated scale and
// a step far from the ends of the exponent range (false for NaN).
template <int FP4>
__device__ __forceinline__ bool common(float a, float s, float step) {
  return s >= 0.015625f && a < 448.0f * Fmt<FP4>::kTop && step > 1e-30f && step < 1e30f;
}

// Any block, by division: x (NaN as 0) -> quotient clamped to the code range.
template <int FP4>
__device__ __forceinline__ float quot_any(float x, float step) {
  const float q = step > 0.0f ? __fdiv_rn(x, step) : 0.0f;
  return fminf(fmaxf(q, -Fmt<FP4>::kTop), Fmt<FP4>::kTop);
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

// ---- K: rows of the half page, two at a time per load instruction
template <int FP4, bool PC>
__device__ __forceinline__ void write_k(const Append4Params& p, uint8_t* half, int kvh, int64_t row0, int lo, int hi,
                                        int lane) {
  const int c = lane & 15, r0 = lane >> 4;   // dims 8c .. 8c+7 of rows r0, r0 + 2, ...
  float g[8], rg[8];
#pragma unroll
  for (int e = 0; e < (PC ? 8 : 1); ++e) {
    g[e] = load_scale(p.k_scale, p.scale_kind, PC ? kvh * kV4Dim + 8 * c + e : kvh);
    rg[e] = rcp_approx(g[e]);
  }
  const __nv_bfloat16* src0 = p.k_new + row0 + (int64_t)kvh * kV4Dim + 8 * c;
  for (int base = lo & ~3; base < hi; base += 4) {
    uint4 x[2];
    bool ok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = base + 2 * i + r0;
      ok[i] = r >= lo && r < hi;
      x[i] = make_uint4(0, 0, 0, 0);
      if (ok[i]) {
        const __nv_bfloat16* src = src0 + (int64_t)(r - lo) * p.kv_stride;
        if (p.vec) {
          x[i] = __ldg(reinterpret_cast<const uint4*>(src));
        } else {
          const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
          x[i] = make_uint4(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16, h[4] | (uint32_t)h[5] << 16,
                            h[6] | (uint32_t)h[7] << 16);
        }
      }
    }
    float f[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[i][2 * e] = bf16_lo(w[e]);
        f[i][2 * e + 1] = bf16_hi(w[e]);
      }
    }
    // the block maxima of both rows; an even lane goes on with row 0's, odd row 1's
    float a;
    bool finite = true;
    {
      uint32_t m[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        m[i] = max_u16x2(max_u16x2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                         max_u16x2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
      uint32_t mm = max_u16x2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
      mm = max_u16x2(mm, __shfl_xor_sync(0xffffffffu, mm, 1));
      const uint32_t mine = (lane & 1) ? mm >> 16 : mm & 0xFFFFu;
      finite = mine < 0x7F80u;
      if constexpr (PC) {
        float y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          y[i] = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i] = fmaxf(y[i], fabsf(__fdiv_rn(f[i][e], g[e])));
        }
        const float t = (lane & 1) ? y[0] : y[1];
        a = fmaxf((lane & 1) ? y[1] : y[0], __shfl_xor_sync(0xffffffffu, t, 1));
      } else {
        a = __fdiv_rn(__uint_as_float(mine << 16), g[0]);
      }
    }
    uint32_t sb = block_scale<FP4>(a);
    float s = e4m3_to_f32(sb);
    const int my_row = base + 2 * (lane & 1) + r0;
    const bool mine_ok = my_row >= lo && my_row < hi;
    uint32_t w[2];
    if (__all_sync(0xffffffffu, !mine_ok || (finite && common<FP4>(a, s, PC ? 1.0f : s * g[0])))) {
      const float st = PC ? s : s * g[0], rs = rcp_approx(st);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float si = __shfl_sync(0xffffffffu, st, (lane & ~1) | i);
        const float ri = __shfl_sync(0xffffffffu, rs, (lane & ~1) | i);
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = PC ? quot(f[i][e], si * g[e], ri * rg[e]) : quot(f[i][e], si, ri);
        w[i] = pack8<FP4>(q);
      }
    } else {
      float y[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        y[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (f[i][e] != f[i][e]) f[i][e] = 0.0f;
          y[i] = fmaxf(y[i], fabsf(__fdiv_rn(f[i][e], g[PC ? e : 0])));
        }
        y[i] = fmaxf(y[i], __shfl_xor_sync(0xffffffffu, y[i], 1));
      }
      sb = block_scale<FP4>((lane & 1) ? y[1] : y[0]);
      s = e4m3_to_f32(sb);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float si = __shfl_sync(0xffffffffu, s, (lane & ~1) | i);
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = quot_any<FP4>(f[i][e], __fmul_rn(si, g[PC ? e : 0]));
        w[i] = pack8<FP4>(q);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (ok[i]) *reinterpret_cast<uint32_t*>(half + (base + 2 * i + r0) * (kV4Dim / 2) + 4 * c) = w[i];
    if (mine_ok) half[kV4Codes + my_row * kV4Nblk + (c >> 1)] = (uint8_t)sb;
  }
}

// ---- V: four dims of every position per lane, eight positions a step
template <int FP4, bool PC>
__device__ __forceinline__ void write_v(const Append4Params& p, uint8_t* half, int kvh, int64_t row0, int lo, int hi,
                                        int lane) {
  const int sub = lane & 3, blk = lane >> 2;
  float g[4], rg[4];
#pragma unroll
  for (int e = 0; e < (PC ? 4 : 1); ++e) {
    g[e] = load_scale(p.v_scale, p.scale_kind, PC ? kvh * kV4Dim + 4 * lane + e : kvh);
    rg[e] = rcp_approx(g[e]);
  }
  const __nv_bfloat16* src0 = p.v_new + row0 + (int64_t)kvh * kV4Dim + 4 * lane;
  uint32_t out[4][4];   // [dim][8-position word]
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int d = 0; d < 4; ++d) out[d][k] = 0;
    if (8 * k + 8 <= lo || 8 * k >= hi) continue;
    uint2 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = 8 * k + j;
      x[j] = make_uint2(0, 0);
      if (r >= lo && r < hi) {
        const __nv_bfloat16* src = src0 + (int64_t)(r - lo) * p.kv_stride;
        if (p.vec) {
          x[j] = __ldg(reinterpret_cast<const uint2*>(src));
        } else {
          const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
          x[j] = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        }
      }
    }
    float q[4][8];   // [dim][position]
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // positions 4h .. 4h+3; lane `sub` works out the scale of 4h + sub
      float f[4][4];   // [position][dim]
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j][0] = bf16_lo(x[4 * h + j].x);
        f[j][1] = bf16_hi(x[4 * h + j].x);
        f[j][2] = bf16_lo(x[4 * h + j].y);
        f[j][3] = bf16_hi(x[4 * h + j].y);
      }
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
      float a;
      if constexpr (PC) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) y[j] = fmaxf(y[j], fabsf(__fdiv_rn(f[j][e], g[e])));
          y[j] = fmaxf(y[j], __shfl_xor_sync(0xffffffffu, y[j], 1));
          y[j] = fmaxf(y[j], __shfl_xor_sync(0xffffffffu, y[j], 2));
        }
        a = (sub & 2) ? ((sub & 1) ? y[3] : y[2]) : ((sub & 1) ? y[1] : y[0]);
      } else {
        a = __fdiv_rn(__uint_as_float(mine << 16), g[0]);
      }
      uint32_t sb = block_scale<FP4>(a);
      float s = e4m3_to_f32(sb);
      const int pos = 8 * k + 4 * h + sub;
      const bool mine_ok = pos >= lo && pos < hi;
      if (__all_sync(0xffffffffu,
                     !mine_ok || (mine < 0x7F80u && common<FP4>(a, s, PC ? 1.0f : s * g[0])))) {
        // (a position outside the range gets finite codes: a word holds several)
        const float st = !mine_ok ? 1.0f : PC ? s : s * g[0], rs = rcp_approx(st);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float sj = __shfl_sync(0xffffffffu, st, (lane & ~3) | j);
          const float rj = __shfl_sync(0xffffffffu, rs, (lane & ~3) | j);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            q[e][4 * h + j] = PC ? quot(f[j][e], sj * g[e], rj * rg[e]) : quot(f[j][e], sj, rj);
        }
      } else {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (f[j][e] != f[j][e]) f[j][e] = 0.0f;
            y[j] = fmaxf(y[j], fabsf(__fdiv_rn(f[j][e], g[PC ? e : 0])));
          }
          y[j] = fmaxf(y[j], __shfl_xor_sync(0xffffffffu, y[j], 1));
          y[j] = fmaxf(y[j], __shfl_xor_sync(0xffffffffu, y[j], 2));
        }
        sb = block_scale<FP4>((sub & 2) ? ((sub & 1) ? y[3] : y[2]) : ((sub & 1) ? y[1] : y[0]));
        s = e4m3_to_f32(sb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float sj = __shfl_sync(0xffffffffu, s, (lane & ~3) | j);
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e][4 * h + j] = quot_any<FP4>(f[j][e], __fmul_rn(sj, g[PC ? e : 0]));
        }
      }
      if (mine_ok) half[kV4Codes + blk * kV4Half + pos] = (uint8_t)sb;
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) out[d][k] = pack8<FP4>(q[d]);
  }
  uint8_t* rows = half + 4 * lane * (kV4Half / 2);
  if (lo == 0 && hi == kV4Half) {
#pragma unroll
    for (int d = 0; d < 4; ++d)
      reinterpret_cast<uint4*>(rows)[d] = make_uint4(out[d][0], out[d][1], out[d][2], out[d][3]);
  } else {
    // part of a half page: the nibbles of other positions stay
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int a = max(0, min(8, lo - 8 * k)), b = max(0, min(8, hi - 8 * k));
      const uint32_t mask = (uint32_t)(((1ull << (4 * b)) - 1) & ~((1ull << (4 * a)) - 1));
      if (mask != 0) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t* w = reinterpret_cast<uint32_t*>(rows + d * (kV4Half / 2)) + k;
          *w = mask == 0xFFFFFFFFu ? out[d][k] : (*w & ~mask) | (out[d][k] & mask);
        }
      }
    }
  }
}

template <int FP4, bool PC>
__global__ void __launch_bounds__(kWarps * 32) cache_append4_kernel(const Append4Params p) {
  const int lane = threadIdx.x & 31;
  const uint32_t id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= p.total) return;
  // side fastest, then kv head: neighbouring warps read neighbouring rows
  const int side = id & 1;
  const uint32_t bu = (id >> 1) / (uint32_t)p.kv_heads;
  const int kvh = (int)((id >> 1) - bu * p.kv_heads);
  const int b = (int)(bu / (uint32_t)p.units), u = (int)(bu % (uint32_t)p.units);
  const int q = p.seq_lens[b];
  if (q <= 0) return;
  const int start = p.seq_lens_kv[b], end = start + q;
  const int h0 = (start / kV4Half + u) * kV4Half;       // first position of the half page
  const int lo = max(h0, start) - h0, hi = min(h0 + kV4Half, end) - h0;
  if (lo >= hi) return;
  const int lp = h0 / kPage;
  const int page = lp < p.max_blocks ? p.block_table[(int64_t)b * p.max_blocks + lp] : -1;
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) record_status(p.status, PA_ERR_BAD_PAGE, b);
    return;
  }
  const int64_t row0 = (int64_t)(p.cu_seqlens_q[b] + (h0 + lo - start)) * p.kv_stride;
  const int64_t off = ((int64_t)page * p.kv_heads + kvh) * kV4Slab + (h0 % kPage) / kV4Half * kV4HalfBytes;
  if (side == 0) write_k<FP4, PC>(p, p.cache_k + off, kvh, row0, lo, hi, lane);
  else write_v<FP4, PC>(p, p.cache_v + off, kvh, row0, lo, hi, lane);
}

}  // namespace

cudaError_t launch_cache_append4(const Plan& plan, const pa_args& a, const void* k_new,
                                 const void* v_new, int64_t kv_stride, int32_t* status,
                                 cudaStream_t stream) {
  const pa_problem& pr = plan.prob;
  if (pr.bsz == 0 || plan.max_q == 0) return cudaSuccess;
  Append4Params p{};
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.kv_stride = kv_stride;
  p.cache_k = static_cast<uint8_t*>(const_cast<void*>(a.cache_k));
  p.cache_v = static_cast<uint8_t*>(const_cast<void*>(a.cache_v));
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.seq_lens_kv = a.seq_lens_kv;
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.status = status;
  p.max_blocks = pr.max_blocks_per_seq;
  p.num_pages = pr.num_pages;
  p.kv_heads = pr.kv_heads;
  p.scale_kind = pr.scale_kind;
  // a range of max_q positions touches at most this many half pages
  p.units = (plan.max_q + kV4Half - 2) / kV4Half + 1;
  p.vec = kv_stride % 8 == 0 && reinterpret_cast<uintptr_t>(k_new) % 16 == 0 &&
          reinterpret_cast<uintptr_t>(v_new) % 16 == 0;
  const double total = 2.0 * pr.bsz * p.units * pr.kv_heads;
  if (total > (double)INT32_MAX) return cudaErrorInvalidValue;
  p.total = (uint32_t)total;
  const uint32_t blocks = (p.total + kWarps - 1) / kWarps;
  const bool pc = pr.scale_kind == PA_SCALE_PER_CHANNEL;
  const dim3 grid(blocks), block(kWarps * 32);
  if (pr.kv_dtype == PA_KV_FP4_E2M1) {
    if (pc) cache_append4_kernel<1, true><<<grid, block, 0, stream>>>(p);
    else cache_append4_kernel<1, false><<<grid, block, 0, stream>>>(p);
  } else {
    if (pc) cache_append4_kernel<0, true><<<grid, block, 0, stream>>>(p);
    else cache_append4_kernel<0, false><<<grid, block, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace pa
