// pa_cache_read.cu - reads a range of cached positions back as bf16 rows: the
// inverse of the cache append, for every cache format.
//
//   value = bf16(stored * scale): 8-bit formats code * scale, 4-bit formats
//   code * (block scale * tensor scale), products in fp32.
//
// One warp per (sequence, half page of 32 positions, kv head, K or V).  K: lane =
// 8 dims of a row, two rows per load and per store instruction.  V (transposed
// in the cache): lane = 4 dims, whose 32 positions it loads as 16-byte runs, so
// that a position's row of 256 bytes leaves as one 8-byte store per lane and no
// transposition is needed.  MLA rows: lane = 8 of 576 dims, three rounds a row.
// What bounds it: the bytes, above all the 2 written per element.
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
  int32_t units;       // half pages a range can touch
  int32_t sides;       // 2 (K, V) or 1 (MLA)
  int32_t vec;         // rows may be written with 16-byte stores
  uint32_t total;      // (sequence, half page, kv head, side) warps
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// N / 2 words of bf16 pairs to dst: one store, or elements where it is not aligned
template <int N>
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, const uint32_t (&w)[N / 2], bool vec) {
  if (vec) {
    if constexpr (N == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      reinterpret_cast<uint16_t*>(dst)[2 * k] = (uint16_t)w[k];
      reinterpret_cast<uint16_t*>(dst)[2 * k + 1] = (uint16_t)(w[k] >> 16);
    }
  }
}

// Two neighbouring codes (4-bit: one byte; 8-bit: two bytes) as fp32, exact.
template <int KV>
__device__ __forceinline__ float2 pair_value(uint32_t b) {
  if constexpr (KV == PA_KV_FP4_E2M1) {
    uint32_t h;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
        : "=r"(h)
        : "r"(b));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
  } else if constexpr (KV == PA_KV_INT4) {
    return make_float2((float)((int)(b << 28) >> 28), (float)((int)(b << 24) >> 28));
  } else if constexpr (KV == PA_KV_FP8_E4M3) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
  } else {
    return make_float2((float)(int8_t)b, (float)(int8_t)(b >> 8));
  }
}

template <int KV>
constexpr bool four() { return KV == PA_KV_INT4 || KV == PA_KV_FP4_E2M1; }

template <int KV, bool PC>
__device__ __forceinline__ void read_k(const ReadParams& p, const uint8_t* slab, int h0, int kvh, int64_t row0, int lo,
                                       int hi, int lane) {
  constexpr bool kFour = four<KV>();
  const int c = lane & 15, r0 = lane >> 4;   // dims 8c .. 8c+7 of rows r0, r0 + 2, ...
  float g[8];
#pragma unroll
  for (int e = 0; e < (PC ? 8 : 1); ++e)
    g[e] = load_scale(p.k_scale, p.scale_kind, PC ? kvh * kV4Dim + 8 * c + e : kvh);
  const uint8_t* half = slab + (kFour ? h0 / kHalf * kV4HalfBytes : h0 * kV4Dim);
  __nv_bfloat16* dst0 = p.k_out + row0 + (int64_t)kvh * kV4Dim + 8 * c;
#pragma unroll 4
  for (int base = lo & ~1; base < hi; base += 2) {
    const int r = base + r0;
    if (r < lo || r >= hi) continue;
    uint32_t w[2] = {0, 0};   // four codes of 8 bits or eight of 4 bits a word
    float bs = 1.0f;
    if constexpr (kFour) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(half + r * (kV4Dim / 2)) + c);
      bs = e4m3_to_f32(__ldg(half + kV4Codes + r * kV4Nblk + (c >> 1)));
    } else {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(half + r * kV4Dim) + c);
      w[0] = x.x;
      w[1] = x.y;
    }
    uint32_t o[4];
    const float step = bs * g[0];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = pair_value<KV>(kFour ? (w[0] >> (8 * k)) & 0xFFu : (w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
      o[k] = bf16_pair(v.x * (PC ? bs * g[2 * k] : step), v.y * (PC ? bs * g[2 * k + 1] : step));
    }
    store_row<8>(dst0 + (int64_t)(r - lo) * p.kv_stride, o, p.vec);
  }
}

template <int KV, bool PC>
__device__ __forceinline__ void read_v(const ReadParams& p, const uint8_t* slab, int h0, int kvh, int64_t row0, int lo,
                                       int hi, int lane) {
  constexpr bool kFour = four<KV>();
  constexpr int kRun = kFour ? 32 : 16;   // positions per 16-byte run of a dim
  float g[4];
#pragma unroll
  for (int e = 0; e < (PC ? 4 : 1); ++e)
    g[e] = load_scale(p.v_scale, p.scale_kind, PC ? kvh * kV4Dim + 4 * lane + e : kvh);
  __nv_bfloat16* dst0 = p.v_out + row0 + (int64_t)kvh * kV4Dim + 4 * lane;
#pragma unroll
  for (int run = 0; run < kHalf / kRun; ++run) {
    const int q0 = run * kRun;   // first position of the run within the half page
    if (q0 >= hi || q0 + kRun <= lo) continue;
    uint4 x[4], s[2];
#pragma unroll
    for (int d = 0; d < 4; ++d)
      x[d] = __ldg(reinterpret_cast<const uint4*>(
          kFour ? slab + h0 / kHalf * kV4HalfBytes + (4 * lane + d) * (kV4Half / 2)
                : slab + (4 * lane + d) * kPage + h0 + q0));
    if constexpr (kFour) {
      const uint8_t* sp = slab + h0 / kHalf * kV4HalfBytes + kV4Codes + (lane >> 2) * kV4Half;
      s[0] = __ldg(reinterpret_cast<const uint4*>(sp));
      s[1] = __ldg(reinterpret_cast<const uint4*>(sp) + 1);
    }
#pragma unroll
    for (int j = 0; j < kRun / 2; ++j) {   // positions q0 + 2j, + 1
      const int pos = q0 + 2 * j;
      if (pos + 1 < lo || pos >= hi) continue;
      float bs[2] = {1.0f, 1.0f};
      if constexpr (kFour) {
        const uint4& sv = s[j >> 3];
        const int wi = (j >> 1) & 3;
        const uint32_t sw = (wi == 0 ? sv.x : wi == 1 ? sv.y : wi == 2 ? sv.z : sv.w) >> (16 * (j & 1));
        const float2 b2 = pair_value<PA_KV_FP8_E4M3>(sw & 0xFFFFu);
        bs[0] = b2.x;
        bs[1] = b2.y;
      }
      float2 v[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int byte = kFour ? j : 2 * j;   // of the 16
        const uint32_t w = (byte >> 2) == 0 ? x[d].x : (byte >> 2) == 1 ? x[d].y : (byte >> 2) == 2 ? x[d].z : x[d].w;
        v[d] = pair_value<KV>((w >> (8 * (byte & 3))) & (kFour ? 0xFFu : 0xFFFFu));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (pos + e < lo || pos + e >= hi) continue;
        const float step = bs[e] * g[0];
        float f[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) f[d] = (e ? v[d].y : v[d].x) * (PC ? bs[e] * g[d] : step);
        const uint32_t o[2] = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])};
        store_row<4>(dst0 + (int64_t)(pos + e - lo) * p.kv_stride, o, p.vec);
      }
    }
  }
}

// MLA: latent rows of head_dim bytes (a multiple of 8), one scale
template <int KV>
__device__ __forceinline__ void read_latent(const ReadParams& p, const uint8_t* page, int h0, int64_t row0, int lo,
                                            int hi, int lane) {
  const float g = load_scale(p.k_scale, PA_SCALE_GLOBAL, 0);
#pragma unroll 4
  for (int r = lo; r < hi; ++r) {
    for (int c = lane; c < p.head_dim / 8; c += 32) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(page + (int64_t)(h0 + r) * p.head_dim) + c);
      const uint32_t w[2] = {x.x, x.y};
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = pair_value<KV>((w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
        o[k] = bf16_pair(v.x * g, v.y * g);
      }
      store_row<8>(p.k_out + row0 + (int64_t)(r - lo) * p.kv_stride + 8 * c, o, p.vec);
    }
  }
}

template <int KV, bool PC>
__global__ void __launch_bounds__(kWarps * 32) cache_read_kernel(const ReadParams p) {
  const int lane = threadIdx.x & 31;
  const uint32_t id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= p.total) return;
  const uint32_t rest = id / (uint32_t)p.sides;
  const int side = (int)(id - rest * p.sides);
  const uint32_t bu = rest / (uint32_t)p.kv_heads;
  const int kvh = (int)(rest - bu * p.kv_heads);
  const int b = (int)(bu / (uint32_t)p.units), u = (int)(bu % (uint32_t)p.units);
  const int q = p.seq_lens[b];
  if (q <= 0) return;
  const int start = p.seq_lens_kv[b], end = start + q;
  const int first = (start / kHalf + u) * kHalf;        // first position of the half page
  const int lo = max(first, start) - first, hi = min(first + kHalf, end) - first;
  if (lo >= hi) return;
  const int lp = first / kPage, h0 = first % kPage;
  const int page = lp < p.max_blocks ? p.block_table[(int64_t)b * p.max_blocks + lp] : -1;
  const int64_t row0 = (int64_t)(p.cu_seqlens_q[b] + (first + lo - start)) * p.kv_stride;
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) record_status(p.status, PA_ERR_BAD_PAGE, b);
    __nv_bfloat16* dst = (side ? p.v_out : p.k_out) + row0 + (int64_t)kvh * p.head_dim;
    for (int r = 0; r < hi - lo; ++r)
      for (int d = lane; d < p.head_dim; d += 32) dst[(int64_t)r * p.kv_stride + d] = __float2bfloat16_rn(0.0f);
    return;
  }
  if constexpr (!four<KV>()) {
    if (p.sides == 1) {
      read_latent<KV>(p, p.cache_k + (int64_t)page * kPage * p.head_dim, h0, row0, lo, hi, lane);
      return;
    }
  }
  const int64_t off = ((int64_t)page * p.kv_heads + kvh) * (four<KV>() ? kV4Slab : kPage * kV4Dim);
  if (side == 0) read_k<KV, PC>(p, p.cache_k + off, h0, kvh, row0, lo, hi, lane);
  else read_v<KV, PC>(p, p.cache_v + off, h0, kvh, row0, lo, hi, lane);
}

template <int KV>
static void launch_kv(const ReadParams& p, uint32_t blocks, cudaStream_t stream) {
  if (p.scale_kind == PA_SCALE_PER_CHANNEL) cache_read_kernel<KV, true><<<blocks, kWarps * 32, 0, stream>>>(p);
  else cache_read_kernel<KV, false><<<blocks, kWarps * 32, 0, stream>>>(p);
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
  // a range of max_q positions touches at most this many half pages
  p.units = (plan.max_q + kHalf - 2) / kHalf + 1;
  p.vec = kv_stride % 8 == 0 && reinterpret_cast<uintptr_t>(k_out) % 16 == 0 &&
          reinterpret_cast<uintptr_t>(p.v_out) % 16 == 0;
  const double total = (double)p.sides * pr.bsz * p.units * pr.kv_heads;
  if (total > (double)INT32_MAX) return cudaErrorInvalidValue;
  p.total = (uint32_t)total;
  const uint32_t blocks = (p.total + kWarps - 1) / kWarps;
  switch (pr.kv_dtype) {
    case PA_KV_INT8: launch_kv<PA_KV_INT8>(p, blocks, stream); break;
    case PA_KV_FP8_E4M3: launch_kv<PA_KV_FP8_E4M3>(p, blocks, stream); break;
    case PA_KV_INT4: launch_kv<PA_KV_INT4>(p, blocks, stream); break;
    default: launch_kv<PA_KV_FP4_E2M1>(p, blocks, stream); break;
  }
  return cudaGetLastError();
}

}  // namespace pa
