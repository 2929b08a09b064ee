// pa_cache4.cu - quantise-and-write of the appended tokens' K / V into the
// 4-bit paged cache: the kernel and its launch (pa_cache4.cuh says what a warp does).
#include "pa_cache4.cuh"

namespace pa {
namespace {

constexpr int kPage = 64;
constexpr int kWarps = 8;
// 64 registers a thread, 32 warps an SM: writing prompts of 31k rows, 8 heads, took 48.6,
// 50.1, 38.2, 43.3 and 49.2 us with 2 to 6 CTAs an SM
constexpr int kCtas = 4;

template <int FP4, bool PC, int U>
__global__ void __launch_bounds__(kWarps * 32, kCtas) cache_append4_kernel(const Append4Params p) {
  const int lane = threadIdx.x & 31;
  const uint32_t id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= p.total) return;
  // side fastest, then kv head: neighbouring warps read neighbouring rows
  const int side = id & 1;
  const uint32_t bu = (id >> 1) / (uint32_t)p.kv_heads;
  const int kvh = (int)((id >> 1) - bu * p.kv_heads);
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
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) record_status(p.status, PA_ERR_BAD_PAGE, b);
    return;
  }
  const __nv_bfloat16* rows = (side ? p.v_new : p.k_new) +
                              (int64_t)(p.cu_seqlens_q[b] + (lo - start)) * p.kv_stride + (int64_t)kvh * kV4Dim;
  uint8_t* half = (side ? p.cache_v : p.cache_k) + ((int64_t)page * p.kv_heads + kvh) * kV4Slab +
                  (u0 % kPage) / kV4Half * kV4HalfBytes;
  const int first = u0 % kV4Half;
  const int a = lo - u0, e = hi - u0;
  // Quotients by pairs, but where their registers are spilled more than they save: a scale a
  // channel, units of 32 (prompts of 1k-8k, 31k rows of 8 heads: int4 67.0 us by pairs, 63.2 one
  // by one, FP4 59.2 and 56.6; units of 8, 8192 rows, both 18.8 and 20.9).
  constexpr bool kPairs = !PC || U < 32;
  if (!p.vec)
    write_any<FP4>(rows, p.kv_stride, side ? p.v_scale : p.k_scale, p.scale_kind, kvh, half, side != 0, first + a,
                   first + e, lane);
  else if (side == 0)
    e - a == U ? write_k<FP4, PC, U, true, kPairs>(p, rows, half, kvh, first, a, e, lane)
               : write_k<FP4, PC, U, false, kPairs>(p, rows, half, kvh, first, a, e, lane);
  else
    e - a == U ? write_v<FP4, PC, U, true, kPairs>(p, rows, half, kvh, first, a, e, lane)
               : write_v<FP4, PC, U, false, kPairs>(p, rows, half, kvh, first, a, e, lane);
}

template <int U>
cudaError_t launch_u(Append4Params& p, const Plan& plan, cudaStream_t stream) {
  const pa_problem& pr = plan.prob;
  p.units = row_units<U>(pr.bsz, plan.max_q, plan.total_q);
  const double total = 2.0 * p.units.count * pr.kv_heads;
  if (total > (double)INT32_MAX) return cudaErrorInvalidValue;
  p.total = (uint32_t)total;
  const dim3 grid((p.total + kWarps - 1) / kWarps), block(kWarps * 32);
  const bool pc = pr.scale_kind == PA_SCALE_PER_CHANNEL;
  if (pr.kv_dtype == PA_KV_FP4_E2M1) {
    if (pc) cache_append4_kernel<1, true, U><<<grid, block, 0, stream>>>(p);
    else cache_append4_kernel<1, false, U><<<grid, block, 0, stream>>>(p);
  } else {
    if (pc) cache_append4_kernel<0, true, U><<<grid, block, 0, stream>>>(p);
    else cache_append4_kernel<0, false, U><<<grid, block, 0, stream>>>(p);
  }
  return cudaGetLastError();
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
  p.vec = kv_stride % 8 == 0 && reinterpret_cast<uintptr_t>(k_new) % 16 == 0 &&
          reinterpret_cast<uintptr_t>(v_new) % 16 == 0;
  // Units of 32 positions; of 8 while those would leave most of the GPU's warps
  // without one (the time of a small call is one warp's walk through its unit)
  return 2.0 * plan.total_q * pr.kv_heads / 32 < 4.0 * kWarps * plan.num_sms
             ? launch_u<8>(p, plan, stream)
             : launch_u<32>(p, plan, stream);
}

}  // namespace pa
