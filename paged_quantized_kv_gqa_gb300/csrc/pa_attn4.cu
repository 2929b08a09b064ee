// pa_attn4.cu - attention over the 4-bit cache, one warp per packed query row.
//
// s_j = sm_scale <q, k_j>, out = sum_j softmax(s)_j v_j over the visible
// positions, with a running maximum and sum in 32 bits.  A CTA takes one work
// item; its warps take the item's rows; lane l holds dims 4l .. 4l+3.
#include <cfloat>

#include "pa_common.cuh"
#include "pa_kv4.cuh"

namespace pa {

template <int FP4>
__global__ void __launch_bounds__(256) attn4_kernel(const uint8_t* __restrict__ ck,
                                                    const uint8_t* __restrict__ cv, const AttnParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Item m = load_item<64>(p.items, blockIdx.x);
  const int G = p.group;
  const int tok0_local = p.attn_mask ? m.tok0 - p.cu_seqlens_q[m.b] : 0;
  const int pre_len = m.cbase - tok0_local;
  const uint8_t* tmask = p.attn_mask ? p.attn_mask + (int64_t)m.b * p.mask_dim * p.mask_dim : nullptr;
  const bool pc = p.scale_kind == PA_SCALE_PER_CHANNEL;
  float gk[4], gv[4];
  for (int e = 0; e < 4; ++e) {
    const int idx = pc ? m.kvh * 128 + 4 * lane + e : m.kvh;
    gk[e] = load_scale(p.k_scale, p.scale_kind, idx);
    gv[e] = load_scale(p.v_scale, p.scale_kind, idx);
  }
  for (int r = warp; r < m.ntok * G; r += blockDim.x / 32) {
    const int token = m.tok0 + r / G, head = m.kvh * G + r % G;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, mx = -INFINITY, l = 0.f;
    for (int e = 0; e < 4; ++e)
      q[e] = __bfloat162float(p.q[(int64_t)token * p.q_stride + (int64_t)head * 128 + 4 * lane + e]) * gk[e];
    const int lim = min(m.kv1, m.cbase + r / G + 1);
    for (int pos = m.kv0; pos < lim; ++pos) {
      if (tmask && pos >= pre_len && !tmask[(tok0_local + r / G) * p.mask_dim + pos - pre_len]) continue;
      const int page = p.block_table[(int64_t)m.b * p.max_blocks + pos / 64];
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) record_status(p.status, PA_ERR_BAD_PAGE, blockIdx.x);
        continue;
      }
      const int64_t slab = ((int64_t)page * p.kv_heads + m.kvh) * kV4Slab;
      const int off = pos % 64;
      const float sk = e4m3_to_f32(ck[slab + k4_scale_off(off, lane / 4)]);
      const float sv = e4m3_to_f32(cv[slab + v4_scale_off(off, lane / 4)]);
      float s = 0.f, v[4];
      for (int e = 0; e < 4; ++e) {
        const uint32_t kb = ck[slab + k4_code_off(off, 4 * lane + e)] >> (4 * (e & 1));
        const uint32_t vb = cv[slab + v4_code_off(off, 4 * lane + e)] >> (4 * (off & 1));
        s += q[e] * (code4_to_f32<FP4>(kb & 15u) * sk);
        v[e] = code4_to_f32<FP4>(vb & 15u) * sv;
      }
      for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      s *= p.sm_scale_log2;
      const float mn = fmaxf(mx, s), a = exp2f(mx - mn), pr = exp2f(s - mn);
      l = l * a + pr;
      for (int e = 0; e < 4; ++e) o[e] = o[e] * a + pr * v[e];
      mx = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f, ln2 = 0.69314718055994530942f;
    const int64_t sp = ((int64_t)token * p.max_chunks + m.chunk) * p.q_heads + head;
    for (int e = 0; e < 4; ++e) {
      const float v = o[e] * inv * gv[e];
      const int d = 4 * lane + e;
      if (m.nch > 1) {
        reinterpret_cast<float*>(p.part_o)[sp * 128 + d] = v;
      } else {
        const float f = ep_value(p.ep, v, head * 128 + d);
        const int64_t oi = ((int64_t)token * p.q_heads + head) * 128 + d;
        if (p.ep.int8_out) reinterpret_cast<int8_t*>(p.out)[oi] = (int8_t)ep_int8(p.ep, f);
        else p.out[oi] = __float2bfloat16_rn(f);
      }
    }
    if (lane == 0) {
      if (m.nch > 1) {
        p.part_m[sp] = l > 0.f ? mx * ln2 : -INFINITY;
        p.part_d[sp] = l;
      } else if (p.lse != nullptr) {
        p.lse[(int64_t)token * p.q_heads + head] = l > 0.f ? (mx + log2f(l)) * ln2 : -INFINITY;
      }
    }
  }
}

cudaError_t launch_attn4(const Plan& plan, const AttnParams& p, const void* ck, const void* cv,
                         cudaStream_t stream) {
  const uint8_t* k = static_cast<const uint8_t*>(ck);
  const uint8_t* v = static_cast<const uint8_t*>(cv);
  if (plan.prob.kv_dtype == PA_KV_FP4_E2M1) attn4_kernel<1><<<plan.num_items(), 256, 0, stream>>>(k, v, p);
  else attn4_kernel<0><<<plan.num_items(), 256, 0, stream>>>(k, v, p);
  return cudaGetLastError();
}

}  // namespace pa
