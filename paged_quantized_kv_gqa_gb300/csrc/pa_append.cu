// pa_append.cu - the 8-bit instantiations of the append kernel (pa_append.cuh).
#include "pa_append.cuh"

namespace pa {

template <int KV>
static cudaError_t launch_t(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                            const CUtensorMap& tm_v, const CUtensorMap& tm_q, cudaStream_t stream) {
  auto kern = append_kernel<KV>;
  const int smem = Smem<false>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<plan.num_ctas, kThreads, smem, stream>>>(tm_k, tm_v, tm_q, nullptr, nullptr, p);
  return cudaGetLastError();
}

cudaError_t launch_append(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                          const CUtensorMap& tm_v, const CUtensorMap& tm_q, cudaStream_t stream) {
  return plan.prob.kv_dtype == PA_KV_FP8_E4M3 ? launch_t<PA_KV_FP8_E4M3>(plan, p, tm_k, tm_v, tm_q, stream)
                                              : launch_t<PA_KV_INT8>(plan, p, tm_k, tm_v, tm_q, stream);
}

}  // namespace pa
