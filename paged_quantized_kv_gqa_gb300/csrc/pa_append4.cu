// pa_append4.cu - the 4-bit instantiations of the append kernel (pa_append.cuh).
#include "pa_append.cuh"

namespace pa {

template <int KV>
static cudaError_t launch_t(const Plan& plan, const AttnParams& p, const uint8_t* ck, const uint8_t* cv,
                            const CUtensorMap& tm_q, cudaStream_t stream) {
  auto kern = append_kernel<KV>;
  const int smem = Smem<true>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<plan.num_ctas, kThreads, smem, stream>>>(tm_q, tm_q, tm_q, ck, cv, p);   // tm_k, tm_v unused
  return cudaGetLastError();
}

cudaError_t launch_append4(const Plan& plan, const AttnParams& p, const void* ck, const void* cv,
                           const CUtensorMap& tm_q, cudaStream_t stream) {
  const uint8_t* k = static_cast<const uint8_t*>(ck);
  const uint8_t* v = static_cast<const uint8_t*>(cv);
  return plan.prob.kv_dtype == PA_KV_FP4_E2M1 ? launch_t<PA_KV_FP4_E2M1>(plan, p, k, v, tm_q, stream)
                                              : launch_t<PA_KV_INT4>(plan, p, k, v, tm_q, stream);
}

}  // namespace pa
