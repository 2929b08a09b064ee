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
#include "pa_common.cuh"
#include "pa_kv4.cuh"

namespace pa {
namespace {

constexpr int kPage = 64;
constexpr int kUnit = 16;   // positions per CTA

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
  int32_t units;       // CTAs per (sequence, kv head)
};

// The block scale of this thread's 16-lane group and the thread's code.
template <int FP4>
__device__ __forceinline__ uint32_t quantise4(float x, float g, uint32_t& scale_byte) {
  constexpr float kTop = FP4 ? 6.0f : 7.0f;
  if (x != x) x = 0.0f;
  float a = fabsf(__fdiv_rn(x, g));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  a = fmaxf(a, 0.0f);   // 0 / 0 of a zero scale
  uint16_t sb;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.0f), "f"(__fdiv_rn(a, kTop)));
  scale_byte = sb & 0xFFu;
  const float step = __fmul_rn(e4m3_to_f32(scale_byte), g);
  float q = step > 0.0f ? __fdiv_rn(x, step) : 0.0f;
  q = fminf(fmaxf(q, -kTop), kTop);
  if constexpr (FP4) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, z;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "mov.b32 %0, {a, a, a, a};\n\t}"
        : "=r"(r)
        : "f"(q), "f"(0.0f));
    return r & 15u;
  } else {
    return (uint32_t)__float2int_rn(q) & 15u;
  }
}

template <int FP4>
__global__ void __launch_bounds__(128) cache_append4_kernel(const Append4Params p) {
  const int b = blockIdx.x / p.units, unit = blockIdx.x % p.units, kvh = blockIdx.y, d = threadIdx.x;
  const int q = p.seq_lens[b];
  if (q <= 0) return;
  const int start = p.seq_lens_kv[b], end = start + q;
  const int u0 = (start / kUnit + unit) * kUnit;
  const int p0 = max(u0, start), p1 = min(u0 + kUnit, end);
  if (p0 >= p1) return;
  const int lp = u0 / kPage;
  const int page = lp < p.max_blocks ? p.block_table[(int64_t)b * p.max_blocks + lp] : -1;
  if (page < 0 || page >= p.num_pages) {
    if (d == 0) record_status(p.status, PA_ERR_BAD_PAGE, b);
    return;
  }
  const int idx = p.scale_kind == PA_SCALE_PER_CHANNEL ? kvh * 128 + d : kvh;
  const float gk = load_scale(p.k_scale, p.scale_kind, idx);
  const float gv = load_scale(p.v_scale, p.scale_kind, idx);
  const int64_t slab = ((int64_t)page * p.kv_heads + kvh) * kV4Slab;
  uint8_t* ck = p.cache_k + slab;
  uint8_t* cv = p.cache_v + slab;
  const int64_t row0 = (int64_t)(p.cu_seqlens_q[b] + (p0 - start)) * p.kv_stride + kvh * 128 + d;
  uint8_t* vrow = cv + v4_code_off(u0 % kPage, d);   // the unit's 8 bytes of this dim
  uint32_t vbyte = 0;
  for (int pos = p0; pos < p1; ++pos) {
    const int64_t src = row0 + (int64_t)(pos - p0) * p.kv_stride;
    const int off = pos % kPage;
    uint32_t sk, sv;
    const uint32_t kc = quantise4<FP4>(__bfloat162float(p.k_new[src]), gk, sk);
    const uint32_t vc = quantise4<FP4>(__bfloat162float(p.v_new[src]), gv, sv);
    const uint32_t kn = __shfl_xor_sync(0xffffffffu, kc, 1);
    if ((d & 1) == 0) ck[k4_code_off(off, d)] = (uint8_t)(kc | (kn << 4));
    if (d % kV4Blk == 0) {
      ck[k4_scale_off(off, d / kV4Blk)] = (uint8_t)sk;
      cv[v4_scale_off(off, d / kV4Blk)] = (uint8_t)sv;
    }
    // a byte holds two positions: a range that starts or ends inside one keeps
    // the other position's nibble
    uint8_t* vb = vrow + (pos - u0) / 2;
    if (pos & 1) {
      *vb = (uint8_t)((pos == p0 ? (*vb & 0x0Fu) : vbyte) | (vc << 4));
    } else {
      vbyte = vc;
      if (pos + 1 == p1) *vb = (uint8_t)((*vb & 0xF0u) | vc);
    }
  }
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
  p.units = (plan.max_q + kUnit - 1) / kUnit + 1;
  if ((int64_t)pr.bsz * p.units > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(pr.bsz * p.units, pr.kv_heads);
  if (pr.kv_dtype == PA_KV_FP4_E2M1) cache_append4_kernel<1><<<grid, 128, 0, stream>>>(p);
  else cache_append4_kernel<0><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
