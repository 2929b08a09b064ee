// pa_cache_read.cu - reads a range of cached positions back as bf16 rows: the
// inverse of the cache append, for every cache format.
//
//   value = bf16(stored * scale): 8-bit formats code * scale, 4-bit formats
//   code * (block scale * tensor scale), products in fp32.
#include "pa_common.cuh"
#include "pa_kv4.cuh"

namespace pa {
namespace {

constexpr int kPage = 64;
constexpr int kUnit = 16;   // positions per CTA

struct ReadParams {
  const uint8_t* cache_k;
  const uint8_t* cache_v;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;       // or null (MLA)
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
  int32_t units;       // CTAs per (sequence, kv head)
};

template <int KV>
__device__ __forceinline__ float stored8(uint32_t b) {
  if constexpr (KV == PA_KV_FP8_E4M3) return e4m3_to_f32(b);
  else return (float)(int8_t)b;
}

template <int KV>
__global__ void __launch_bounds__(128) cache_read_kernel(const ReadParams p) {
  constexpr bool kFour = KV == PA_KV_INT4 || KV == PA_KV_FP4_E2M1;
  const int b = blockIdx.x / p.units, unit = blockIdx.x % p.units, kvh = blockIdx.y;
  const int q = p.seq_lens[b];
  if (q <= 0) return;
  const int start = p.seq_lens_kv[b], end = start + q;
  const int u0 = (start / kUnit + unit) * kUnit;
  const int p0 = max(u0, start), p1 = min(u0 + kUnit, end);
  if (p0 >= p1) return;
  const int lp = u0 / kPage;
  const int page = lp < p.max_blocks ? p.block_table[(int64_t)b * p.max_blocks + lp] : -1;
  const bool ok = page >= 0 && page < p.num_pages;
  if (!ok && threadIdx.x == 0) record_status(p.status, PA_ERR_BAD_PAGE, b);
  for (int d = threadIdx.x; d < p.head_dim; d += blockDim.x) {
    const int idx = p.scale_kind == PA_SCALE_PER_CHANNEL ? kvh * p.head_dim + d : kvh;
    const float gk = load_scale(p.k_scale, p.scale_kind, idx);
    const float gv = p.v_out ? load_scale(p.v_scale, p.scale_kind, idx) : 0.0f;
    for (int pos = p0; pos < p1; ++pos) {
      const int off = pos % kPage;
      float k = 0.0f, v = 0.0f;
      if (ok) {
        if constexpr (kFour) {
          const int64_t slab = ((int64_t)page * p.kv_heads + kvh) * kV4Slab;
          const uint8_t *ck = p.cache_k + slab, *cv = p.cache_v + slab;
          constexpr int F = KV == PA_KV_FP4_E2M1;
          const uint32_t kb = ck[k4_code_off(off, d)] >> (4 * (d & 1));
          const uint32_t vb = cv[v4_code_off(off, d)] >> (4 * (off & 1));
          k = code4_to_f32<F>(kb & 15u) * (e4m3_to_f32(ck[k4_scale_off(off, d / kV4Blk)]) * gk);
          v = code4_to_f32<F>(vb & 15u) * (e4m3_to_f32(cv[v4_scale_off(off, d / kV4Blk)]) * gv);
        } else {
          const int64_t slab = (int64_t)page * p.kv_heads + kvh;
          k = stored8<KV>(p.cache_k[(slab * kPage + off) * p.head_dim + d]) * gk;
          if (p.v_out) v = stored8<KV>(p.cache_v[(slab * p.head_dim + d) * kPage + off]) * gv;
        }
      }
      const int64_t dst = (int64_t)(p.cu_seqlens_q[b] + pos - start) * p.kv_stride + (int64_t)kvh * p.head_dim + d;
      p.k_out[dst] = __float2bfloat16_rn(k);
      if (p.v_out) p.v_out[dst] = __float2bfloat16_rn(v);
    }
  }
}

}  // namespace

cudaError_t launch_cache_read(const Plan& plan, const pa_args& a, void* k_out, void* v_out,
                              int64_t kv_stride, int32_t* status, cudaStream_t stream) {
  const pa_problem& pr = plan.prob;
  if (pr.bsz == 0 || plan.max_q == 0) return cudaSuccess;
  ReadParams p{};
  p.cache_k = static_cast<const uint8_t*>(a.cache_k);
  p.cache_v = static_cast<const uint8_t*>(a.cache_v);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = pr.layout == PA_LAYOUT_MLA ? nullptr : static_cast<__nv_bfloat16*>(v_out);
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
  p.units = (plan.max_q + kUnit - 1) / kUnit + 1;
  if ((int64_t)pr.bsz * p.units > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(pr.bsz * p.units, pr.kv_heads);
  switch (pr.kv_dtype) {
    case PA_KV_INT8: cache_read_kernel<PA_KV_INT8><<<grid, 128, 0, stream>>>(p); break;
    case PA_KV_FP8_E4M3: cache_read_kernel<PA_KV_FP8_E4M3><<<grid, 128, 0, stream>>>(p); break;
    case PA_KV_INT4: cache_read_kernel<PA_KV_INT4><<<grid, 128, 0, stream>>>(p); break;
    default: cache_read_kernel<PA_KV_FP4_E2M1><<<grid, 128, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace pa
