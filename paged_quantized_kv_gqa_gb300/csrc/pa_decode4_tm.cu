// pa_decode4_tm.cu - the instantiations of the tensor-memory decode kernel of the 4-bit
// cache (pa_decode.cuh); tiles of at most 16 rows run in pa_decode4.cu.
#include "pa_decode.cuh"

namespace pa {

template <int NR, int KV>
static cudaError_t launch_t(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                            const uint8_t* cv, cudaStream_t stream) {
  const bool pc = p.scale_kind == PA_SCALE_PER_CHANNEL;
  auto kern = p.attn_mask != nullptr ? (pc ? decode_kernel<NR, KV, true, true> : decode_kernel<NR, KV, true, false>)
                                     : (pc ? decode_kernel<NR, KV, false, true> : decode_kernel<NR, KV, false, false>);
  const int smem = Smem<NR>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<plan.num_ctas, kThreads, smem, stream>>>(tm_k, cv, p);
  return cudaGetLastError();
}

template <int NR>
static cudaError_t launch_nr(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                             const uint8_t* cv, cudaStream_t stream) {
  return plan.prob.kv_dtype == PA_KV_FP4_E2M1 ? launch_t<NR, PA_KV_FP4_E2M1>(plan, p, tm_k, cv, stream)
                                              : launch_t<NR, PA_KV_INT4>(plan, p, tm_k, cv, stream);
}

cudaError_t launch_decode4_tm(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                              const void* cv, cudaStream_t stream) {
  const uint8_t* v = static_cast<const uint8_t*>(cv);
  switch (plan.decode_rows) {
    case 32: return launch_nr<32>(plan, p, tm_k, v, stream);
    case 48: return launch_nr<48>(plan, p, tm_k, v, stream);
    case 64: return launch_nr<64>(plan, p, tm_k, v, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
