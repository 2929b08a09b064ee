// pa_merge.cu - split-KV partial-state merge and the raw-gather test hook.
//
// Merge (FastDeploy append_attention_c8_impl.cuh, merge_multi_chunks_*_kernel
// launched after the split kernel; the arithmetic is in pa_merge.cuh).
// 8-bit plans: one warp per (token, query head); the partial states of a token sit
// at slot (token * max_chunks + c) * q_heads + head.  4-bit and expanded plans: one warp per eight
// chunks; the states at (first slot of the token + c) * q_heads + head, the
// slots numbered without gaps.  HBM-bound, CUDA cores: the row reads of all chunks are
// issued before they are summed.
#include <algorithm>
#include <cfloat>

#include "pa_common.cuh"
#include "pa_index.cuh"
#include "pa_merge.cuh"

namespace pa {

// One row whose chunk count is at most kPre: the (m, d) loads and every chunk
// row's loads go out in a single round (the row loads do not depend on the
// weights), so the row costs one memory round trip instead of three.
template <int DV, int kPre>
__device__ __forceinline__ void merge_row_short(const __nv_bfloat16* __restrict__ part_o,
                                                const float* __restrict__ part_m,
                                                const float* __restrict__ part_d, int64_t slot0,
                                                int64_t cstride, int nch, int lane,
                                                float (&acc)[DV / 32], float& M, float& W) {
  constexpr int kPer = DV / 32;
  constexpr int kVecBytes = (kPer % 8 == 0) ? 16 : 8;
  constexpr int kVec = kPer * 2 / kVecBytes;
  float mc = -INFINITY, dc = 0.f;
  if (lane < nch) {
    mc = __ldcg(part_m + slot0 + lane * cstride);
    dc = __ldcg(part_d + slot0 + lane * cstride);
  }
  uint4 raw[kPre][kVec];
#pragma unroll
  for (int c = 0; c < kPre; ++c) {
    const __nv_bfloat16* src = part_o + (slot0 + c * cstride) * DV + lane * kPer;
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      raw[c][k] = make_uint4(0u, 0u, 0u, 0u);
      if (c < nch) {
        if constexpr (kVecBytes == 16) {
          raw[c][k] = __ldcg(reinterpret_cast<const uint4*>(src) + k);
        } else {
          const uint2 h = __ldcg(reinterpret_cast<const uint2*>(src) + k);
          raw[c][k].x = h.x;
          raw[c][k].y = h.y;
        }
      }
    }
  }
  M = mc;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  W = 0.f;
  if (M == -INFINITY) return;
  const float w = (mc != -INFINITY) ? dc * __expf(mc - M) : 0.f;
  W = w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
#pragma unroll
  for (int c = 0; c < kPre; ++c) {
    const float wc = __shfl_sync(0xffffffffu, w, c);
    if (c < nch && wc != 0.f) {
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        const uint32_t wd[4] = {raw[c][k].x, raw[c][k].y, raw[c][k].z, raw[c][k].w};
#pragma unroll
        for (int e = 0; e < kVecBytes / 4; ++e) {
          const __nv_bfloat162 b2 = *reinterpret_cast<const __nv_bfloat162*>(&wd[e]);
          acc[k * (kVecBytes / 2) + 2 * e + 0] += wc * __low2float(b2);
          acc[k * (kVecBytes / 2) + 2 * e + 1] += wc * __high2float(b2);
        }
      }
    }
  }
}

// 512-wide rows: five blocks per SM, so that a 128-head MLA batch's rows are
// merged in one wave
template <int DV>
__global__ void __launch_bounds__(256, DV >= 512 ? 5 : 1) merge_kernel(const int32_t* __restrict__ merge_tokens,
                                                    const int32_t* __restrict__ nch_token,
                                                    int n_merge, int q_heads, int max_chunks,
                                                    const __nv_bfloat16* __restrict__ part_o,
                                                    const float* __restrict__ part_m,
                                                    const float* __restrict__ part_d,
                                                    void* __restrict__ out,
                                                    float* __restrict__ lse,
                                                    const OutEpilogue ep) {
  pdl_wait();   // launched as a programmatic dependent of the attention kernel
  const int wid = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= n_merge * q_heads) return;
  const int token = merge_tokens[wid / q_heads];
  const int head = wid % q_heads;
  const int nch = nch_token[token];
  const int64_t slot0[1] = {(int64_t)token * max_chunks * q_heads + head};
  float acc[1][DV / 32], M[1], W[1];
  // 128-wide rows with at most 8 chunks: one round of loads (512-wide rows keep
  // the register budget that gives five blocks per SM)
  bool done = false;
  if constexpr (DV < 512) {
    if (nch <= 8) {
      merge_row_short<DV, 8>(part_o, part_m, part_d, slot0[0], q_heads, nch, lane, acc[0], M[0], W[0]);
      done = true;
    }
  }
  if (!done) {
    const bool valid[1] = {true};
    merge_rows<DV, 1>(part_o, part_m, part_d, slot0, valid, q_heads, nch, lane, acc, M, W);
  }
  // 512-wide rows are MLA's, whose out is 16-byte aligned: the branch for other addresses
  // cost an MLA step 0.6 of the 8.3 us outside its attention kernel (means of seven runs)
  merge_store<DV, (DV < 512)>(acc[0], M[0], W[0], out, lse, ep, token, head, q_heads, lane);
}

// Rows whose partial states are fp32 (plans over a 4-bit cache or expanded rows), 128 wide, lane l
// owning dims 4l .. 4l+3 (one 16-byte load per chunk row).  Warp w of a row takes
// chunks 8 w .. 8 w + 7, then those 8 * (warps of the row) further on; its first eight
// rows are requested before the weights are known, so that a row of at most eight
// chunks a warp costs one memory round trip after its entry's lookup.  The warps' sums
// meet in shared memory.  A row without chunks comes out as 0, -inf.
//   merge_f32_kernel          every row gets the warps that the longest one takes
//   merge_f32_classes_kernel  a row gets the warps that its own chunks take.  The plan's
//                             entries come in classes by their chunks, a block of 32
//                             warps works on one class.
// The first is used while all rows are of one class or its warps fit the GPU at once
// (the lookup of the classes costs 0.6 us).  Beyond that it is what the call waits for:
// one sequence of 131k positions beside 255 of 500, 64 heads, had 9280 rows merged by
// 262144 warps, 153 us; by their own 10 us.
struct MergeGrid {
  uint32_t block[kMergeClasses + 1];   // first block of each class; the grid's size
  uint32_t entry[kMergeClasses + 1];   // first entry of each class; their count
};

// One row by `wpr` warps of the block, of which this is warp `sub` (all of them call it).
__device__ __forceinline__ void merge_f32_row(const int4 entry, bool valid, int head, int q_heads, int wpr, int sub,
                                              int warp, int lane, float4 (*sums)[32], float* weights,
                                              const float* __restrict__ part_o, const float* __restrict__ part_m,
                                              const float* __restrict__ part_d, void* __restrict__ out,
                                              float* __restrict__ lse, const OutEpilogue& ep) {
  constexpr int kU = 8;
  const int token = entry.x, nch = entry.y;
  const int64_t slot0 = (int64_t)entry.z * q_heads + head;
  const float4* rows = reinterpret_cast<const float4*>(part_o) + slot0 * 32 + lane;
  const int64_t rstride = (int64_t)q_heads * 32;
  float4 v[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int c = kU * sub + u;
    v[u] = c < nch ? __ldcg(rows + c * rstride) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float M = -INFINITY;
  for (int c = lane; c < nch; c += 32) M = fmaxf(M, __ldcg(part_m + slot0 + (int64_t)c * q_heads));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, W = 0.f;
  if (M != -INFINITY) {
    for (int c0 = kU * sub; c0 < nch; c0 += kU * wpr) {
      if (c0 != kU * sub) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
          v[u] = c0 + u < nch ? __ldcg(rows + (c0 + u) * rstride) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float w = 0.f;   // lane u: weight of chunk c0 + u
      if (lane < kU && c0 + lane < nch) {
        const float m = __ldcg(part_m + slot0 + (int64_t)(c0 + lane) * q_heads);
        if (m != -INFINITY) w = __ldcg(part_d + slot0 + (int64_t)(c0 + lane) * q_heads) * __expf(m - M);
      }
      W += w;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const float wc = __shfl_sync(0xffffffffu, w, u);
        if (wc != 0.f) {
          acc[0] += wc * v[u].x;
          acc[1] += wc * v[u].y;
          acc[2] += wc * v[u].z;
          acc[3] += wc * v[u].w;
        }
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
    W = __shfl_sync(0xffffffffu, W, 0);
  }
  if (wpr > 1) {   // (the same for the whole block)
    sums[warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if (lane == 0) weights[warp] = W;
    __syncthreads();
    if (sub != 0) return;
#pragma unroll 4
    for (int k = 1; k < wpr; ++k) {
      const float4 t = sums[warp + k][lane];
      acc[0] += t.x;
      acc[1] += t.y;
      acc[2] += t.z;
      acc[3] += t.w;
      W += weights[warp + k];
    }
  }
  if (valid) merge_store<128>(acc, M, W, out, lse, ep, token, head, q_heads, lane);
}


template <int WPR>
__global__ void __launch_bounds__(WPR <= 8 ? 256 : 32 * WPR)
    merge_f32_kernel(const int4* __restrict__ merge_rows, int n_merge, int q_heads, const float* __restrict__ part_o,
                     const float* __restrict__ part_m, const float* __restrict__ part_d, void* __restrict__ out,
                     float* __restrict__ lse, const OutEpilogue ep) {
  constexpr int kBlockWarps = WPR <= 8 ? 8 : WPR;
  __shared__ float4 sums[kBlockWarps][32];
  __shared__ float weights[kBlockWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t row = blockIdx.x * (kBlockWarps / WPR) + warp / WPR;
  const bool valid = row < (uint32_t)n_merge * (uint32_t)q_heads;
  // (the plan's arrays were there before the attention kernel started)
  const int4 entry = valid ? merge_rows[row / (uint32_t)q_heads] : make_int4(0, 0, 0, 0);
  const int head = valid ? (int)(row % (uint32_t)q_heads) : 0;
  pdl_wait();   // launched as a programmatic dependent of the attention kernel
  merge_f32_row(entry, valid, head, q_heads, WPR, warp % WPR, warp, lane, sums, weights, part_o, part_m, part_d, out,
                lse, ep);
}

__global__ void __launch_bounds__(1024)
    merge_f32_classes_kernel(const int4* __restrict__ merge_rows, const MergeGrid grid, int q_heads,
                             const float* __restrict__ part_o, const float* __restrict__ part_m,
                             const float* __restrict__ part_d, void* __restrict__ out, float* __restrict__ lse,
                             const OutEpilogue ep) {
  __shared__ float4 sums[32][32];
  __shared__ float weights[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int lw = kMergeClasses - 1;   // 2^lw warps a row in this block's class
  uint32_t block = blockIdx.x, at = 0, end = grid.entry[1];
#pragma unroll
  for (int c = 1; c < kMergeClasses; ++c)
    if (blockIdx.x >= grid.block[c]) {
      lw = kMergeClasses - 1 - c;
      block = blockIdx.x - grid.block[c];
      at = grid.entry[c];
      end = grid.entry[c + 1];
    }
  const uint32_t row = block * (32u >> lw) + (uint32_t)(warp >> lw);
  at += row / (uint32_t)q_heads;
  const bool valid = at < end;
  const int4 entry = valid ? merge_rows[at] : make_int4(0, 0, 0, 0);
  pdl_wait();
  merge_f32_row(entry, valid, (int)(row % (uint32_t)q_heads), q_heads, 1 << lw, warp & ((1 << lw) - 1), warp, lane,
                sums, weights, part_o, part_m, part_d, out, lse, ep);
}

cudaError_t launch_merge(const Plan& plan, const WsView& ws, void* out, float* lse,
                         const OutEpilogue& ep, cudaStream_t stream) {
  const int n_merge = (int)plan.merge_tokens.size();
  if (n_merge == 0) return cudaSuccess;
  const int64_t warps = (int64_t)n_merge * plan.prob.q_heads;
  if (warps > INT32_MAX / 32) return cudaErrorInvalidValue;
  const int blocks = (int)((warps + 7) / 8);
  // programmatic dependent launch: the grid is set up while the attention
  // kernel's last CTAs finish, and waits for it in pdl_wait
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int32_t* mt = ws.merge_tokens;
  const int32_t* nt = ws.nch_token;
  const int qh = plan.prob.q_heads, mc = plan.max_chunks;
  const __nv_bfloat16* po = ws.part_o;
  const float* pm = ws.part_m;
  const float* pd = ws.part_d;
  if (plan.compact()) {
    const float* pf = reinterpret_cast<const float*>(po);
    const int32_t* cls = plan.merge_class;
    int longest = 0;   // its class
    while (cls[longest] == cls[longest + 1]) ++longest;
    const int wpr = 1 << (kMergeClasses - 1 - longest);
    if (cls[longest + 1] < n_merge && warps * wpr > 32 * (int64_t)plan.num_sms) {
      MergeGrid grid;
      int64_t total = 0;
      for (int c = 0; c < kMergeClasses; ++c) {
        grid.block[c] = (uint32_t)total;
        grid.entry[c] = (uint32_t)cls[c];
        const int64_t per_block = 32 >> (kMergeClasses - 1 - c);   // rows
        total += ((int64_t)(cls[c + 1] - cls[c]) * qh + per_block - 1) / per_block;
      }
      grid.block[kMergeClasses] = (uint32_t)total;
      grid.entry[kMergeClasses] = (uint32_t)n_merge;
      cfg.gridDim = dim3((unsigned)total);
      cfg.blockDim = dim3(1024);
      return cudaLaunchKernelEx(&cfg, merge_f32_classes_kernel, ws.merge_rows, grid, qh, pf, pm, pd, out, lse, ep);
    }
    const int block_warps = std::max(8, wpr);
    cfg.gridDim = dim3((unsigned)((warps * wpr + block_warps - 1) / block_warps));
    cfg.blockDim = dim3(32 * block_warps);
    auto kern = wpr == 1   ? merge_f32_kernel<1>
                : wpr == 2 ? merge_f32_kernel<2>
                : wpr == 4 ? merge_f32_kernel<4>
                : wpr == 8 ? merge_f32_kernel<8>
                : wpr == 16 ? merge_f32_kernel<16>
                            : merge_f32_kernel<32>;
    return cudaLaunchKernelEx(&cfg, kern, ws.merge_rows, n_merge, qh, pf, pm, pd, out, lse, ep);
  }
  if (plan.prob.head_dim_v == 128)
    return cudaLaunchKernelEx(&cfg, merge_kernel<128>, mt, nt, n_merge, qh, mc, po, pm, pd, out, lse, ep);
  if (plan.prob.head_dim_v == 512)
    return cudaLaunchKernelEx(&cfg, merge_kernel<512>, mt, nt, n_merge, qh, mc, po, pm, pd, out, lse, ep);
  return cudaErrorInvalidValue;
}

// ------------------------------------------------------------------ gather
__global__ void gather_kernel(const uint8_t* __restrict__ cache_k, const uint8_t* __restrict__ cache_v,
                              const int32_t* __restrict__ block_table, int max_blocks, int num_pages,
                              int kv_heads, int page_size, int dqk, int dv, int mla, int b, int kvh,
                              int pos0, int n, uint8_t* __restrict__ dk, uint8_t* __restrict__ dv_out) {
  const int k = blockIdx.x;
  if (k >= n) return;
  const int pos = pos0 + k;
  const int page = page_of(block_table, max_blocks, b, pos, page_size);
  const int off = pos % page_size;
  const bool ok = page >= 0 && page < num_pages;
  for (int e = threadIdx.x; e < dqk; e += blockDim.x) {
    uint8_t v = 0;
    if (ok) {
      v = mla ? cache_k[((int64_t)page * page_size + off) * dqk + e]
              : cache_k[(((int64_t)page * kv_heads + kvh) * page_size + off) * dqk + e];
    }
    dk[(int64_t)k * dqk + e] = v;
  }
  for (int e = threadIdx.x; e < dv; e += blockDim.x) {
    uint8_t v = 0;
    if (ok) {
      v = mla ? cache_k[((int64_t)page * page_size + off) * dqk + e]
              : cache_v[(((int64_t)page * kv_heads + kvh) * dv + e) * page_size + off];
    }
    dv_out[(int64_t)k * dv + e] = v;
  }
}

cudaError_t launch_gather(const pa_problem& prob, const pa_args& a, int32_t b, int32_t kvh,
                          int32_t pos0, int32_t n, void* dk, void* dv, cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  gather_kernel<<<n, 128, 0, stream>>>(
      static_cast<const uint8_t*>(a.cache_k), static_cast<const uint8_t*>(a.cache_v),
      a.block_table, prob.max_blocks_per_seq, prob.num_pages, prob.kv_heads, prob.block_size,
      prob.head_dim_qk, prob.head_dim_v, prob.layout == PA_LAYOUT_MLA ? 1 : 0, b, kvh, pos0, n,
      static_cast<uint8_t*>(dk), static_cast<uint8_t*>(dv));
  return cudaGetLastError();
}

}  // namespace pa
