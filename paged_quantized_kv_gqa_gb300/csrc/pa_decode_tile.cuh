// pa_decode_tile.cuh - what the tensor-memory decode kernels of the 8-bit cache
// (pa_decode.cu) and of the 4-bit cache (pa_decode.cuh) share: tile sizes, the row
// reductions over a warp, a CTA's item records and its walk over their tiles.
#pragma once

#include "pa_common.cuh"

namespace pa {
namespace {

constexpr int kTileTok = 128;
constexpr int kHeadDim = 128;
constexpr int kPage = 64;
constexpr float kTau = 8.0f;                     // lazy-rescale threshold (log2 units)
constexpr uint32_t kTmemCols = 512;
constexpr int kPBufs = 4;                        // P^T ring depth
// P^T buffer: [128 positions][64 rows] fp16, MN-major (rows contiguous),
// 128-byte swizzle; a thread (= position) writes its rows with 16-byte stores
constexpr int kPBufBytes = kTileTok * 128;
// Item records and per-kv-head scales kept in shared memory: every role reads
// them at each item boundary, where a read from memory would wait behind the
// kernel's own page stream.
constexpr int kCachedItems = 160;
constexpr int kCachedHeads = 64;

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// The decode pipeline is latency-bound: its waits re-probe every 32 ns.
__device__ __forceinline__ bool dwait(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                      volatile int* abort_any) {
  return wait_or_abort(bar, parity, limit_ns, abort_any, 32);
}

// Sums n values per thread (one per row) over the 32 lanes of a warp, all rows
// at once.  While n is even, each exchange sends half of the rows still held to
// the partner lane and keeps the other half (the lane with the offset bit set
// keeps the upper half), so the warp spends n/2 + n/4 + ... shuffles instead of
// 5 n; once n is odd the remaining offsets exchange everything.  On return v[0
// .. left) holds the sums of rows row0 .. row0 + left - 1, and the lanes that
// differ only in the bits of the full exchanges hold the same values.
template <int N, int O>
__device__ __forceinline__ void sum_rows_step(float* v, int lane, int& row0) {
  if constexpr (N % 2 == 0 && N > 1) {
    constexpr int H = N / 2;
    const bool up = (lane & O) != 0;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const float send = up ? v[k] : v[k + H];
      const float keep = up ? v[k + H] : v[k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, O);
    }
    if (up) row0 += H;
    if constexpr (O > 1) sum_rows_step<H, O / 2>(v, lane, row0);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], O);
    if constexpr (O > 1) sum_rows_step<N, O / 2>(v, lane, row0);
  }
}

// The same exchange for the row maxima.  The first step reads the tile's
// values and writes half as many, so that they stay intact for the softmax.
template <int N, int O>
__device__ __forceinline__ void max_rows_step(float* v, int lane, int& row0) {
  if constexpr (N % 2 == 0 && N > 1) {
    constexpr int H = N / 2;
    const bool up = (lane & O) != 0;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const float send = up ? v[k] : v[k + H];
      const float keep = up ? v[k + H] : v[k];
      v[k] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, O));
    }
    if (up) row0 += H;
    if constexpr (O > 1) max_rows_step<H, O / 2>(v, lane, row0);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = fmaxf(v[k], __shfl_xor_sync(0xffffffffu, v[k], O));
    if constexpr (O > 1) max_rows_step<N, O / 2>(v, lane, row0);
  }
}
template <int N>
__device__ __forceinline__ void max_rows_first(const float* s, float* t, int lane, int& row0) {
  constexpr int H = N / 2;
  const bool up = (lane & 16) != 0;
#pragma unroll
  for (int k = 0; k < H; ++k) {
    const float send = up ? s[k] : s[k + H];
    const float keep = up ? s[k + H] : s[k];
    t[k] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 16));
  }
  if (up) row0 += H;
  max_rows_step<H, 8>(t, lane, row0);
}

// rows one lane holds after sum_rows_step<N, 16>
template <int N, int O = 16>
constexpr int sum_rows_left() {
  if constexpr (O == 0) return N;
  else if constexpr (N % 2 == 0 && N > 1) return sum_rows_left<N / 2, O / 2>();
  else return sum_rows_left<N, O / 2>();
}

// Page-stage ring depth.  Three stages measured faster than four at every
// row count (48 rows: 1.56-1.65 -> 1.527 ms on spec-verify-4; 32 rows 0.611
// -> 0.601 ms): the copies still run well ahead of the converter.
constexpr int kPageStages = 3;

// TMEM columns: K[2] 0/64, V[2] 128/192, S[2] 256/256+NR, O[2] 256+2NR/256+3NR.
template <int NR>
struct Tm {
  static constexpr uint32_t K0 = 0, V0 = 128, S0 = 256, O0 = 256 + 2 * NR;
  static_assert(256 + 4 * NR <= 512, "TMEM overflow");
};

// The CTA's item records: the first kCachedItems from shared memory.
template <bool FOUR>   // records of a plan over a 4-bit cache
struct ItemSrc {
  const int32_t* cached;   // shared memory
  const int32_t* items;    // global
  int begin, n_cached;
  __device__ __forceinline__ Item at(int it) const {
    const int k = it - begin;
    if (k < n_cached) {
      const int4* r = reinterpret_cast<const int4*>(cached + k * kItemWords);
      return FOUR ? item4_from<kTileTok>(r[0], r[1]) : item_from<kTileTok>(r[0], r[1]);
    }
    return FOUR ? load_item4<kTileTok>(items, it) : load_item<kTileTok>(items, it);
  }
};

// Walks the (item, tile) sequence of one CTA.
template <bool FOUR>
struct TileCursor {
  int it, end, i, ntiles;
  ItemSrc<FOUR> src;
  __device__ __forceinline__ void init(const ItemSrc<FOUR>& s, int begin, int e) {
    src = s;
    it = begin;
    end = e;
    i = 0;
    ntiles = it < end ? src.at(it).ntiles : 0;
  }
  __device__ __forceinline__ bool valid() const { return it < end; }
  __device__ __forceinline__ void advance() {
    if (++i >= ntiles) {
      ++it;
      i = 0;
      ntiles = it < end ? src.at(it).ntiles : 0;
    }
  }
};

}  // namespace
}  // namespace pa
