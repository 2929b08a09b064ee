// pa_kv4.cuh - the 4-bit cache: slab layout, code and scale conversions.
//
// K and V of one (page, kv head) are a slab each: two half pages of 32
// positions one after the other, so that a half page (what a warp works on) is
// one contiguous, 16-byte aligned run of bytes and moves with one bulk copy:
//   K half  codes  [32 positions][64 bytes]   byte i = dims 2i (low nibble), 2i+1
//           scales [32 positions][8]          E4M3, one per 16 dims
//   V half  codes  [128 dims][16 bytes]       byte i = positions 2i (low), 2i+1
//           scales [8 blocks of 16 dims][32 positions]
// V is transposed (as in the 8-bit cache) so that an MMA operand's pairs along
// the positions are neighbours; its scales are transposed with it.
//
// A stored value is code * block scale * tensor scale.  code * block scale has
// at most 3 + 4 significant bits and lies in [2^-10, 3584], so it is exact in
// fp16: the attention kernels multiply in fp16 without a rounding, and the
// tensor scale enters where the 8-bit kernels apply theirs (per channel K: into
// Q'; otherwise into the softmax scale; V: at the output).
#pragma once

#include <cstdint>

#include "pa.h"
#include "pa_ptx.cuh"

namespace pa {

constexpr int kV4Half = 32;                              // positions per half page
constexpr int kV4Dim = 128;
constexpr int kV4Blk = 16;                               // dims per block scale
constexpr int kV4Nblk = kV4Dim / kV4Blk;
constexpr int kV4Codes = kV4Half * kV4Dim / 2;           // code bytes of a half page
constexpr int kV4HalfBytes = kV4Codes + kV4Half * kV4Nblk;
constexpr int kV4Slab = 2 * kV4HalfBytes;                // one (page, kv head) of K or V
static_assert(kV4HalfBytes % 16 == 0, "half pages move with bulk copies");

// byte offsets within a slab; pos = position within the page
__device__ __forceinline__ int k4_code_off(int pos, int dim) {
  return (pos / kV4Half) * kV4HalfBytes + (pos % kV4Half) * (kV4Dim / 2) + dim / 2;
}
__device__ __forceinline__ int k4_scale_off(int pos, int blk) {
  return (pos / kV4Half) * kV4HalfBytes + kV4Codes + (pos % kV4Half) * kV4Nblk + blk;
}
__device__ __forceinline__ int v4_code_off(int pos, int dim) {
  return (pos / kV4Half) * kV4HalfBytes + dim * (kV4Half / 2) + (pos % kV4Half) / 2;
}
__device__ __forceinline__ int v4_scale_off(int pos, int blk) {
  return (pos / kV4Half) * kV4HalfBytes + kV4Codes + blk * kV4Half + pos % kV4Half;
}

// E4M3 byte -> fp32 (exact)
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(b & 0xFF)));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFF)));
}

// a 4-bit code -> fp32 (exact).  FP4: E2M1, sign in bit 3; else two's complement.
template <int FP4>
__device__ __forceinline__ float code4_to_f32(uint32_t c) {
  if constexpr (FP4) {
    uint32_t h;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
        : "=r"(h)
        : "r"(c & 15u));
    return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFF)));
  } else {
    return (float)((int)(c << 28) >> 28);
  }
}

// The units of U positions that ranges of rows touch, for kernels with one warp per
// unit (and kv head, and side).  Numbering them as bsz rectangles of the longest
// range's count leaves most warps without work when one prompt is written beside
// many single tokens (8192 rows beside 255 of 1, 8 kv heads: 418 us, with the other
// numbering 18.2), but needs no search (writing 16 prompts of up to 4k rows: 67.7 us
// for the pair of calls, 68.0 with it), so it is used up to twice the numbers of the
// other.  That gives sequence b the numbers from cu[b] / U + 2 b on: a range of q
// rows touches at most q / U + 2 units, whatever its start.  A warp finds its
// sequence by a search of 32 ways a step (one step up to 32 sequences, two up to 1024).
struct RowUnits {
  int32_t per_seq;   // units of a rectangle; 0: by search
  int32_t bsz;
  int64_t count;     // numbers given out
};

inline RowUnits row_units_of(int U, int bsz, int max_q, int64_t total_q) {
  const int per_seq = (max_q + U - 2) / U + 1;   // touched at most by a range of max_q rows
  const int64_t rect = (int64_t)bsz * per_seq, by_rows = total_q / U + 2 * (int64_t)bsz;
  return rect <= 2 * by_rows ? RowUnits{per_seq, bsz, rect} : RowUnits{0, bsz, by_rows};
}

template <int U>
inline RowUnits row_units(int bsz, int max_q, int64_t total_q) {
  return row_units_of(U, bsz, max_q, total_q);
}

// Unit number n -> sequence and unit of its range (a number may be past the range's
// last unit); the whole warp calls it.  Units of 1 << shift.
__device__ __forceinline__ void find_unit_of(int shift, const RowUnits& ru, const int32_t* cu, uint32_t n, int lane, int& b,
                                             int& u) {
  if (ru.per_seq > 0) {
    b = (int)(n / (uint32_t)ru.per_seq);
    u = (int)(n - (uint32_t)b * (uint32_t)ru.per_seq);
    return;
  }
  auto first = [&](int k) { return ((uint32_t)cu[k] >> shift) + 2u * (uint32_t)k; };
  int lo = 0, hi = ru.bsz;   // first(lo) <= n < first(hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, k = lo + lane * step;
    const int at = __popc(__ballot_sync(0xffffffffu, k < hi && first(k) <= n));   // true for the first lanes
    lo += (max(at, 1) - 1) * step;
    hi = min(hi, lo + step);
  }
  b = lo;
  u = (int)(n - first(lo));
}

template <int U>
__device__ __forceinline__ void find_unit(const RowUnits& ru, const int32_t* cu, uint32_t n, int lane, int& b, int& u) {
  static_assert((U & (U - 1)) == 0, "a power of two");
  constexpr int shift = U == 1 ? 0 : U == 2 ? 1 : U == 4 ? 2 : U == 8 ? 3 : U == 16 ? 4 : U == 32 ? 5 : 6;
  static_assert(1 << shift == U, "up to 64");
  find_unit_of(shift, ru, cu, n, lane, b, u);
}

// Eight codes of a word -> four fp16x2 words, in the order `codes8` defines:
//   FP4   word i = codes (2i, 2i + 1): one hardware conversion per byte;
//   int4  word i = codes (i, i + 4), as 1024 + (code + 8) for even i and
//         64 + (code + 8) for odd i: the nibble, its sign bit flipped, in the
//         mantissa of that power of two (one logic operation per pair, one
//         shift per word).
// scaled() makes code * scale of it, exact in fp16 (see the file comment).
template <int FP4>
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&o)[4]) {
  if constexpr (FP4) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
  } else {
    const uint32_t u = w >> 8;
    o[0] = (w & 0x000F000Fu) ^ 0x64086408u;
    o[1] = (w & 0x00F000F0u) ^ 0x54805480u;
    o[2] = (u & 0x000F000Fu) ^ 0x64086408u;
    o[3] = (u & 0x00F000F0u) ^ 0x54805480u;
  }
}

template <int FP4>
__device__ __forceinline__ uint32_t scaled(uint32_t x, uint32_t s, int i) {
  uint32_t r;
  if constexpr (!FP4)   // 1032 and 72
    asm("sub.f16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"((i & 1) ? 0x54805480u : 0x64086408u));
  asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(s));
  return r;
}

// The first element of pair i and the distance to its second, in elements, where
// eight neighbours unpack to four fp16x2 words (8-bit formats: in order).
template <int KV>
__host__ __device__ constexpr int pair_first(int i) {
  return KV == PA_KV_INT4 ? 8 * (i / 4) + i % 4 : 2 * i;
}
template <int KV>
__host__ __device__ constexpr int pair_gap() {
  return KV == PA_KV_INT4 ? 4 : 1;
}

// Eight E4M3 scales -> four fp16x2 words in the order of codes8.
template <int FP4>
__device__ __forceinline__ void scales8(uint2 w, uint32_t (&o)[4]) {
  if constexpr (FP4) {
    e4m3x4_to_f16x4(w.x, o[0], o[1]);
    e4m3x4_to_f16x4(w.y, o[2], o[3]);
  } else {
    e4m3x4_to_f16x4(__byte_perm(w.x, w.y, 0x5140), o[0], o[1]);
    e4m3x4_to_f16x4(__byte_perm(w.x, w.y, 0x7362), o[2], o[3]);
  }
}

// Keeps the first n of eight scale bytes (n may be negative or above 8).
__device__ __forceinline__ void keep_scales(uint2& w, int n) {
  if (n < 8) {
    w.x = n <= 0 ? 0u : n >= 4 ? w.x : w.x & (0xFFFFFFFFu >> (8 * (4 - n)));
    w.y = n <= 4 ? 0u : w.y & (0xFFFFFFFFu >> (8 * (8 - n)));
  }
}

// One half of an fp16x2 word twice: written as moves, which become an operand's half
// selection in the instruction that uses it (as byte permutations they took the
// integer pipe, the busiest one: batch of 64, int4, 46.8 us, so 45.5).
__device__ __forceinline__ uint32_t lo2(uint32_t h) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tmov.b32 %0, {a, a};\n\t}" : "=r"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t hi2(uint32_t h) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tmov.b32 %0, {b, b};\n\t}" : "=r"(r) : "r"(h));
  return r;
}

// Two E4M3 scales -> each as an fp16x2 word of two equal halves.
__device__ __forceinline__ void scale_pair(uint16_t b, uint32_t& s0, uint32_t& s1) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(b));
  s0 = lo2(h);
  s1 = hi2(h);
}

// One instruction instead of scaled()'s two, where a scale serves enough codes to
// pay for its constants: (2^k + code + 8) * (s / 8) - (2^k + 8) * (s / 8) as one
// fused multiply-add.  Exact for int4: the offset's product is 129 s or 9 s, at
// most 11 significant bits below 57800, and the result is code * s / 8.  The
// caller multiplies what it sums by kFold8.
template <int FP4>
constexpr float kFold8 = FP4 ? 1.f : 8.f;

__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// f16x2 of scales -> s / 8 and the offsets of codes8's even and odd words
__device__ __forceinline__ void fold8(uint32_t h, uint32_t& s, uint32_t& n_even, uint32_t& n_odd) {
  s = mul_h2(h, 0x30003000u);        // 1 / 8
  n_even = mul_h2(h, 0xD808D808u);   // -129
  n_odd = mul_h2(h, 0xC880C880u);    // -9
}

template <int FP4>
__device__ __forceinline__ uint32_t scaled_fold8(uint32_t x, uint32_t s, uint32_t n) {
  if constexpr (FP4) return mul_h2(x, s);
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(s), "r"(n));
  return r;
}

// Two E4M3 scales -> per scale, as words of two equal halves: what scaled_fold8
// takes (FP4: the scale alone).
template <int FP4>
__device__ __forceinline__ void scale_pair_fold8(uint16_t b, uint32_t (&s)[2], uint32_t (&n)[2][2]) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(b));
  if constexpr (!FP4) {
    uint32_t e, o;
    fold8(h, h, e, o);
    n[0][0] = lo2(e);
    n[0][1] = lo2(o);
    n[1][0] = hi2(e);
    n[1][1] = hi2(o);
  }
  s[0] = lo2(h);
  s[1] = hi2(h);
}

}  // namespace pa
