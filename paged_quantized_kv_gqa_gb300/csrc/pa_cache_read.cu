// pa_cache_read.cu - reads a range of cached positions back as bf16 rows: the
// inverse of the cache append, for every cache format.
//
//   value = bf16(stored * scale): 8-bit formats code * scale, 4-bit formats
//   code * (block scale * tensor scale), products in fp32.
//
// One warp per (sequence, unit of 32 or 8 positions, kv head, K or V).  K: lane =
// 8 dims of a row, two rows per load and per store instruction.  V (transposed
// in the cache): lane = 4 dims, whose positions it loads as runs of bytes, so
// that a position's row of 256 bytes leaves as one 8-byte store per lane and no
// transposition is needed.  Rows that are not aligned go position by position.  MLA rows:
// lane = 8 of 576 dims, three rounds a row.
// What bounds it: the bytes, above all the 2 written per element (88k rows of 8
// heads, FP4, in 74.0 us: 0.92 of the copy bandwidth).
#include "pa_common.cuh"
#include "pa_kv4.cuh"

namespace pa {
namespace {

constexpr int kPage = 64;
constexpr int kWarps = 8;
constexpr int kHalf = 32;

struct ReadParams {
  const uint8_t* cache_k;
  const uint8_t* cache_v;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int64_t kv_stride;
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
  int32_t head_dim;
  int32_t scale_kind;
  RowUnits units;
  int32_t sides;       // 2 (K, V) or 1 (MLA)
  int32_t vec;         // rows may be written with 16-byte stores
  uint32_t total;      // (sequence, unit, kv head, side) warps
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// One stored code as fp32.
template <int KV>
__device__ __forceinline__ float one_value(uint32_t b) {
  if constexpr (KV == PA_KV_INT8) return (float)(int8_t)b;
  else if constexpr (KV == PA_KV_FP8_E4M3) return e4m3_to_f32(b);
  else return code4_to_f32<KV == PA_KV_FP4_E2M1>(b & 15u);
}

template <int KV>
constexpr bool four() { return KV == PA_KV_INT4 || KV == PA_KV_FP4_E2M1; }

// Eight stored codes (4-bit: w[0]; 8-bit: both words) as fp32, in order.
template <int KV>
__device__ __forceinline__ void values8(const uint32_t (&w)[2], float (&f)[8]) {
  uint32_t h[4];
  if constexpr (four<KV>()) {
    codes8<KV == PA_KV_FP4_E2M1>(w[0], h);
    if constexpr (KV == PA_KV_INT4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = scaled<0>(h[i], 0x3C003C00u, i);   // times 1
    }
  } else {
    cvt4<KV == PA_KV_FP8_E4M3>(w[0], h[0], h[1]);
    cvt4<KV == PA_KV_FP8_E4M3>(w[1], h[2], h[3]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[pair_first<KV>(i)] = v.x;
    f[pair_first<KV>(i) + pair_gap<KV>()] = v.y;
  }
}

// ---- any positions [lo, hi) of the page's half, any alignment: lane = 4 dims
template <int KV>
__device__ __noinline__ void read_any(__nv_bfloat16* dst, int64_t stride, const void* scale, int kind, int kvh,
                                      const uint8_t* slab, int h0, bool value_side, int lo, int hi, int lane) {
  constexpr bool kFour = four<KV>();
  float g[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    g[e] = load_scale(scale, kind, kind == PA_SCALE_PER_CHANNEL ? kvh * kV4Dim + 4 * lane + e : kvh);
  dst += 4 * lane;
#pragma unroll 1
  for (int r = h0 + lo; r < h0 + hi; ++r, dst += stride) {
    float bs = 1.0f;
    if constexpr (kFour)
      bs = e4m3_to_f32(slab[value_side ? v4_scale_off(r, lane >> 2) : k4_scale_off(r, lane >> 2)]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 4 * lane + e;
      uint32_t b;
      if constexpr (kFour)
        b = value_side ? slab[v4_code_off(r, d)] >> (4 * (r & 1)) : slab[k4_code_off(r, d)] >> (4 * (d & 1));
      else
        b = slab[value_side ? d * kPage + r : r * kV4Dim + d];
      dst[e] = __float2bfloat16_rn(one_value<KV>(b) * (bs * g[e]));
    }
  }
}

// ---- K, positions [lo, hi) of the unit of U that starts at `first` of the half
// page (FULL: all of them; the others' bytes are read, not written); rows: the row
// of position lo
template <int KV, bool PC, int U, bool FULL>
__device__ __forceinline__ void read_k(const ReadParams& p, __nv_bfloat16* rows, const uint8_t* slab, int h0, int kvh,
                                       int first, int lo, int hi, int lane) {
  constexpr bool kFour = four<KV>();
  const int c = lane & 15, r0 = lane >> 4;   // dims 8c .. 8c+7 of rows r0, r0 + 2, ...
  float g[8];
#pragma unroll
  for (int e = 0; e < (PC ? 8 : 1); ++e)
    g[e] = load_scale(p.k_scale, p.scale_kind, PC ? kvh * kV4Dim + 8 * c + e : kvh);
  const uint8_t* half = slab + (kFour ? h0 / kHalf * kV4HalfBytes : h0 * kV4Dim);
  const uint8_t* codes = half + (first + r0) * (kFour ? kV4Dim / 2 : kV4Dim) + (kFour ? 4 : 8) * c;
  const uint8_t* scales = half + kV4Codes + (first + r0) * kV4Nblk + (c >> 1);
  __nv_bfloat16* dst = rows + (FULL ? r0 : r0 - lo) * p.kv_stride + 8 * c;
  constexpr int kB = 4;   // rows in flight per lane
#pragma unroll
  for (int base = 0; base < U; base += 2 * kB) {
    uint32_t w[kB][2], sb[kB];
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const int r = base + 2 * i;
      if constexpr (kFour) {
        w[i][0] = __ldg(reinterpret_cast<const uint32_t*>(codes + r * (kV4Dim / 2)));
        sb[i] = __ldg(scales + r * kV4Nblk);
      } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(codes + r * kV4Dim));
        w[i][0] = x.x;
        w[i][1] = x.y;
      }
    }
#pragma unroll
    for (int i = 0; i < kB; ++i, dst += 2 * p.kv_stride) {
      const float bs = kFour ? e4m3_to_f32(sb[i]) : 1.0f, step = bs * g[0];
      float f[8];
      values8<KV>(w[i], f);
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o[k] = bf16_pair(f[2 * k] * (PC ? bs * g[2 * k] : step), f[2 * k + 1] * (PC ? bs * g[2 * k + 1] : step));
      const int r = base + 2 * i + r0;
      if (FULL || (r >= lo && r < hi)) *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ---- V, the same
template <int KV, bool PC, int U, bool FULL>
__device__ __forceinline__ void read_v(const ReadParams& p, __nv_bfloat16* rows, const uint8_t* slab, int h0, int kvh,
                                       int first, int lo, int hi, int lane) {
  constexpr bool kFour = four<KV>();
  float g[4];
#pragma unroll
  for (int e = 0; e < (PC ? 4 : 1); ++e)
    g[e] = load_scale(p.v_scale, p.scale_kind, PC ? kvh * kV4Dim + 4 * lane + e : kvh);
  const uint8_t* half = slab + h0 / kHalf * kV4HalfBytes;   // 4-bit
  // 16 positions a step where the unit has them (8-bit: a 16-byte run), else 8
  constexpr int kN = U >= 16 ? 16 : 8;
  __nv_bfloat16* dst = rows - (FULL ? 0 : lo * p.kv_stride) + 4 * lane;
#pragma unroll
  for (int q0 = 0; q0 < U; q0 += kN) {
    constexpr int kW = kFour ? kN / 8 : kN / 4;   // words of a dim
    uint32_t w[4][kW], sc[kN / 4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          kFour ? half + (4 * lane + d) * (kV4Half / 2) + (first + q0) / 2
                : slab + (4 * lane + d) * kPage + h0 + first + q0);
      if constexpr (kW == 4) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(src));
        w[d][0] = x.x, w[d][1] = x.y, w[d][2] = x.z, w[d][3] = x.w;
      } else if constexpr (kW == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
        w[d][0] = x.x, w[d][1] = x.y;
      } else {
        w[d][0] = __ldg(src);
      }
    }
    if constexpr (kFour) {
      const uint8_t* sp = half + kV4Codes + (lane >> 2) * kV4Half + first + q0;
#pragma unroll
      for (int k = 0; k < kN / 8; ++k) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(sp) + k);
        sc[2 * k] = x.x;
        sc[2 * k + 1] = x.y;
      }
    }
#pragma unroll
    for (int k = 0; k < kN / 8; ++k) {   // eight positions
      float f[4][8], bs[8];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t x[2] = {w[d][kFour ? k : 2 * k], w[d][kFour ? k : 2 * k + 1]};
        values8<KV>(x, f[d]);
      }
      if constexpr (kFour) {
        const uint32_t x[2] = {sc[2 * k], sc[2 * k + 1]};
        values8<PA_KV_FP8_E4M3>(x, bs);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j, dst += p.kv_stride) {
        const float b = kFour ? bs[j] : 1.0f, step = b * g[0];
        float o[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = f[d][j] * (PC ? b * g[d] : step);
        const int r = q0 + 8 * k + j;
        if (FULL || (r >= lo && r < hi))
          *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3]));
      }
    }
  }
}

// MLA: latent rows of head_dim bytes (a multiple of 8), one scale
template <int KV>
__device__ __forceinline__ void read_latent(const ReadParams& p, __nv_bfloat16* rows, const uint8_t* codes, int n,
                                            int lane) {
  const float g = load_scale(p.k_scale, PA_SCALE_GLOBAL, 0);
#pragma unroll 4
  for (int r = 0; r < n; ++r) {
    for (int c = lane; c < p.head_dim / 8; c += 32) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(codes + r * p.head_dim) + c);
      const uint32_t w[2] = {x.x, x.y};
      float f[8];
      values8<KV>(w, f);
      __nv_bfloat16* dst = rows + r * p.kv_stride + 8 * c;
      if (p.vec) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(bf16_pair(f[0] * g, f[1] * g), bf16_pair(f[2] * g, f[3] * g),
                                                    bf16_pair(f[4] * g, f[5] * g), bf16_pair(f[6] * g, f[7] * g));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[e] = __float2bfloat16_rn(f[e] * g);
      }
    }
  }
}

template <int KV, bool PC, int U>
__global__ void __launch_bounds__(kWarps * 32) cache_read_kernel(const ReadParams p) {
  const int lane = threadIdx.x & 31;
  const uint32_t id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= p.total) return;
  const uint32_t rest = id / (uint32_t)p.sides;
  const int side = (int)(id - rest * p.sides);
  const uint32_t bu = rest / (uint32_t)p.kv_heads;
  const int kvh = (int)(rest - bu * p.kv_heads);
  int b, u;
  find_unit<U>(p.units, p.cu_seqlens_q, bu, lane, b, u);
  const int q = p.seq_lens[b];
  if (q <= 0) return;
  const int start = p.seq_lens_kv[b], end = start + q;
  const int u0 = (start / U + u) * U;                   // first position of the unit
  const int lo = max(u0, start), hi = min(u0 + U, end);
  if (lo >= hi) return;
  const int lp = u0 / kPage;
  const int page = lp < p.max_blocks ? p.block_table[(int64_t)b * p.max_blocks + lp] : -1;
  __nv_bfloat16* rows = (side ? p.v_out : p.k_out) + (int64_t)(p.cu_seqlens_q[b] + (lo - start)) * p.kv_stride +
                        (int64_t)kvh * p.head_dim;
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) record_status(p.status, PA_ERR_BAD_PAGE, b);
    for (int r = 0; r < hi - lo; ++r)
      for (int d = lane; d < p.head_dim; d += 32) rows[r * p.kv_stride + d] = __float2bfloat16_rn(0.0f);
    return;
  }
  if constexpr (!four<KV>()) {
    if (p.sides == 1) {
      read_latent<KV>(p, rows, p.cache_k + ((int64_t)page * kPage + lo % kPage) * p.head_dim, hi - lo, lane);
      return;
    }
  }
  const uint8_t* slab = (side ? p.cache_v : p.cache_k) +
                        ((int64_t)page * p.kv_heads + kvh) * (four<KV>() ? kV4Slab : kPage * kV4Dim);
  const int h0 = u0 % kPage / kHalf * kHalf, first = u0 % kHalf;
  const int a = lo - u0, e = hi - u0;
  if (!p.vec)
    read_any<KV>(rows, p.kv_stride, side ? p.v_scale : p.k_scale, p.scale_kind, kvh, slab, h0, side != 0, first + a,
                 first + e, lane);
  else if (side == 0)
    e - a == U ? read_k<KV, PC, U, true>(p, rows, slab, h0, kvh, first, a, e, lane)
               : read_k<KV, PC, U, false>(p, rows, slab, h0, kvh, first, a, e, lane);
  else
    e - a == U ? read_v<KV, PC, U, true>(p, rows, slab, h0, kvh, first, a, e, lane)
               : read_v<KV, PC, U, false>(p, rows, slab, h0, kvh, first, a, e, lane);
}

template <int KV, int U>
cudaError_t launch_u(ReadParams& p, const Plan& plan, cudaStream_t stream) {
  p.units = row_units<U>(plan.prob.bsz, plan.max_q, plan.total_q);
  const double total = (double)p.sides * p.units.count * plan.prob.kv_heads;
  if (total > (double)INT32_MAX) return cudaErrorInvalidValue;
  p.total = (uint32_t)total;
  const uint32_t blocks = (p.total + kWarps - 1) / kWarps;
  if (p.scale_kind == PA_SCALE_PER_CHANNEL) cache_read_kernel<KV, true, U><<<blocks, kWarps * 32, 0, stream>>>(p);
  else cache_read_kernel<KV, false, U><<<blocks, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

// Units of 32 positions; of 8 while those would leave most of the GPU's warps
// without one (the time of a small call is one warp's walk through its unit).
template <int KV>
cudaError_t launch_kv(ReadParams& p, const Plan& plan, cudaStream_t stream) {
  return (double)p.sides * plan.total_q * plan.prob.kv_heads / 32 < 4.0 * kWarps * plan.num_sms
             ? launch_u<KV, 8>(p, plan, stream)
             : launch_u<KV, 32>(p, plan, stream);
}

}  // namespace

cudaError_t launch_cache_read(const Plan& plan, const pa_args& a, void* k_out, void* v_out,
                              int64_t kv_stride, int32_t* status, cudaStream_t stream) {
  const pa_problem& pr = plan.prob;
  if (pr.bsz == 0 || plan.max_q == 0) return cudaSuccess;
  const bool mla = pr.layout == PA_LAYOUT_MLA;
  ReadParams p{};
  p.cache_k = static_cast<const uint8_t*>(a.cache_k);
  p.cache_v = static_cast<const uint8_t*>(a.cache_v);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = mla ? nullptr : static_cast<__nv_bfloat16*>(v_out);
  p.kv_stride = kv_stride;
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
  p.head_dim = pr.head_dim_qk;
  p.scale_kind = pr.scale_kind;
  p.sides = mla ? 1 : 2;
  p.vec = kv_stride % 8 == 0 && reinterpret_cast<uintptr_t>(k_out) % 16 == 0 &&
          reinterpret_cast<uintptr_t>(p.v_out) % 16 == 0;
  switch (pr.kv_dtype) {
    case PA_KV_INT8: return launch_kv<PA_KV_INT8>(p, plan, stream);
    case PA_KV_FP8_E4M3: return launch_kv<PA_KV_FP8_E4M3>(p, plan, stream);
    case PA_KV_INT4: return launch_kv<PA_KV_INT4>(p, plan, stream);
    default: return launch_kv<PA_KV_FP4_E2M1>(p, plan, stream);
  }
}

}  // namespace pa
