// pa_decode.cu - the 8-bit instantiations of the tensor-memory decode kernel
// (pa_decode.cuh).
#include "pa_decode.cuh"

namespace pa {

template <int NR, int KV>
static cudaError_t launch_t(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                            const CUtensorMap& tm_v, cudaStream_t stream) {
  // the tree-mask variant is a separate instantiation so that the plain
  // causal path carries none of its registers
  auto kern = p.attn_mask != nullptr ? decode_kernel<NR, KV, true> : decode_kernel<NR, KV, false>;
  const int smem = Smem<NR>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<plan.num_ctas, Roles<KV>::kThreads, smem, stream>>>(tm_k, tm_v, nullptr, p);
  return cudaGetLastError();
}

template <int NR>
static cudaError_t launch_nr(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                             const CUtensorMap& tm_v, cudaStream_t stream) {
  return plan.prob.kv_dtype == PA_KV_FP8_E4M3 ? launch_t<NR, PA_KV_FP8_E4M3>(plan, p, tm_k, tm_v, stream)
                                              : launch_t<NR, PA_KV_INT8>(plan, p, tm_k, tm_v, stream);
}

cudaError_t launch_decode(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                          const CUtensorMap& tm_v, cudaStream_t stream) {
  switch (plan.decode_rows) {
    case 16: return launch_nr<16>(plan, p, tm_k, tm_v, stream);
    case 32: return launch_nr<32>(plan, p, tm_k, tm_v, stream);
    case 48: return launch_nr<48>(plan, p, tm_k, tm_v, stream);
    case 64: return launch_nr<64>(plan, p, tm_k, tm_v, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
