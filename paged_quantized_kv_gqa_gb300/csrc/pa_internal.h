// pa_internal.h - structures shared by the host API and the kernel launchers.
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>
#include <vector>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pa.h"

namespace pa {

constexpr int kItemWords = 8;        // b, kvh, token0, n_tok, causal_base, kv0, kv1, c|nch<<16
constexpr int kDecodeRows = 64;      // packed (token, head) rows per decode tile
constexpr int kWarpDecodeRows = 16;  // decode tiles up to this many rows run warp per item
constexpr int kAppendRows = 256;     // packed rows per append item (two 128-row tiles)
// Warps of a 4-bit decode CTA (each takes whole items): up to 8 rows, and 9 to 16, which
// need twice the accumulators.  Plans cut for as many: cut for 16, plans of 9 to 16 rows
// took 77.5 us (32 sequences of 2-8k, 16 rows, int4; for 8 68.4), 35.6 (24 of up to 3k; 26.0)
// and 228 (8 of 32k-131k; 219).
constexpr int decode4_warps(int rows) { return rows <= 8 ? 16 : 8; }
// 4-bit decode plans keep their tiles whole while none is longer: up to there the
// merge's launch costs more than the split saves
constexpr int kDecode4WholePages = 8;
constexpr int kDecode4MinPages = 2;  // smallest share of a warp
constexpr int kDecode4MinTiles = 4;  // smallest share of a tensor-memory CTA, 128-position tiles
// What starting and ending a piece costs, in half pages of a warp and of a CTA.
// With shares of equal pages (cost 0) the warps with the most pieces finished last
// (24 sequences of up to 3k positions 22.0 us, at 2 20.6).  Warps: 30 batches of random
// lengths, five of each of six shapes (16 to 100 sequences of up to 1.5-9k, 1 to 8 rows),
// took 248.2, 245.5, 246.9 and 249.5 us at costs of 1 to 4, summed over the shapes; a
// single batch moves by 5 % either way with the cuts.  CTAs: 6 drafts after 32 prefixes
// of up to 32k positions 311.6, at 8 308.9, at 12 and 16 308.0.
constexpr int kDecode4ItemCost = 2;
constexpr int kDecode4TileCost = 12;
// the merge's classes of 4-bit rows: 32, 16, 8, 4, 2, 1 warps a row, for more than 128,
// 64, 32, 16, 8 chunks and the others
constexpr int kMergeClasses = 6;
// Tiles of 256 rows and a head from which CTA pairs expand (pa_mla_expand.cu; below, a CTA a
// tile of 128 rows): at 256 tiles (333 rows, 128 heads) 22.8 us against 18.9, at 512 (1024
// rows, 128 heads; 8192 rows, 16) 33.2 against 43.3 and 31.2 against 41.8
constexpr int kExpandPairTiles = 384;
constexpr int kExpandedTile = 128;   // positions of a step of the expanded form
// A block of heads that the expanded form's plans keep together: the bytes of its keys and
// values, so that the tiles of a head find them in L2 (129 MB)
constexpr int64_t kExpandedBlock = 48ll << 20;
constexpr int kSlab4 = 4608;         // bytes of one (page, kv head) of a 4-bit K or V cache
constexpr int kStatusBytes = 256;    // status block at the start of the workspace
constexpr int64_t kDefaultWaitNs = 2000000000LL;
constexpr int64_t kMinWaitNs = 1000000LL;      // floor of the test hook's wait limit

// Status block layout (int32 words): [0] status code, [1] detail, [2] cta, [3] spare.

struct Plan {
  pa_problem prob{};
  int32_t family = 0;
  int32_t chunk = 0;
  int32_t tokens_per_tile = 0;
  int32_t num_ctas = 0;
  int32_t total_q = 0;
  int32_t max_chunks = 1;
  int32_t num_sms = 0;
  int32_t decode_rows = 0;    // padded row count (decode family)
  int32_t max_q = 0;          // longest query run (appended tokens per sequence)
  std::vector<int32_t> items;        // [n][8] CTA-major
  std::vector<int32_t> work_indptr;  // [num_ctas+1]
  std::vector<int32_t> nch_token;    // [T]
  std::vector<int32_t> merge_tokens; // [n_merge]
  // split rows of a decode-family plan are merged inside the attention kernel
  // (the CTA that finishes a row group's last chunk merges it); pa_merge is
  // then a no-op
  bool fused_merge = false;
  // a plan made with chunk_size 0 promises rows that need no pa_merge: where it has
  // rows for the merge all the same (4-bit decode, cross attention to nothing), pa_run
  // enqueues the merge kernel itself and pa_merge is a no-op
  bool merge_in_run() const { return prob.chunk_size == 0 && !merge_tokens.empty(); }
  // device blob = work_indptr | items | nch_token | merge_tokens | merge
  // counters [total_q][kv_heads] (zeros; fused merge only) (int32), at
  // kStatusBytes; each array starts at a multiple of 4 words (16 bytes).
  // Plans over a 4-bit cache: item records as item4_from (pa_common.cuh) reads them,
  // and in place of the merge tokens an entry {token, chunks, its first slot, 0} each,
  // class by class.
  std::vector<int32_t> blob;
  size_t off_indptr = 0, off_items = 0, off_nch = 0, off_merge = 0, off_cnt = 0;  // int32 offsets
  size_t plan_bytes = 0;
  size_t part_o_off = 0, part_m_off = 0, part_d_off = 0, ws_bytes = 0;  // byte offsets
  // 4-bit plans: slots of all partial rows (a slot holds q_heads rows); the chunks of
  // a token are neighbours, tokens in order, those with one chunk or none left out
  int64_t part_slots = 0;
  int32_t merge_class[kMergeClasses + 1] = {};   // first merge entry of each class
  int64_t kv_bytes = 0;
  double flops = 0.0;
  // rows of split ranges are fp32 in slots numbered without gaps, the merge by classes
  bool compact() const { return four_bit() || expanded(); }
  bool expanded() const { return prob.layout == PA_LAYOUT_MLA_EXPANDED; }
  int64_t kv_rows = 0;   // expanded rows of all sequences
  bool four_bit() const { return prob.kv_dtype == PA_KV_INT4 || prob.kv_dtype == PA_KV_FP4_E2M1; }
  int32_t num_items() const { return (int32_t)(items.size() / kItemWords); }
};

// Device pointers derived from a workspace.
struct WsView {
  int32_t* status;
  const int32_t* work_indptr;
  const int32_t* items;
  const int32_t* nch_token;
  const int32_t* merge_tokens;
  int32_t* merge_cnt;   // fused merge counters or null
  const int4* merge_rows;   // 4-bit plans: entries in place of the merge tokens
  __nv_bfloat16* part_o;   // fp32 rows for 4-bit plans
  float* part_m;
  float* part_d;
};

struct FaultCfg {
  int64_t wait_limit_ns;
  int32_t skip_first_load;
  uint64_t* trace;        // device timeline buffer or null
  int32_t trace_ctas;
  int32_t trace_tiles;
  int32_t fused_merge;    // plans built while 1 merge decode split rows in-kernel (default 0)
};

// Output epilogue applied where a query row's final output is written
// (FastDeploy append_attention_c8_impl.cuh: shift_bias / smooth_weight
// [q_heads * Dv] and the int8 output with in_scale and the quant bounds):
//   v' = (v + shift) * smooth;  bf16(v') or int8 clamp(rint(v' * q_scale), q_min, q_max)
// with q_scale = quant_max_bound * in_scale.  Split rows apply it in the merge.
struct OutEpilogue {
  const __nv_bfloat16* shift;    // or null
  const __nv_bfloat16* smooth;   // or null
  int32_t int8_out;
  float q_scale, q_min, q_max;
};

// Kernel parameter block for the attention kernels (passed by value).
struct AttnParams {
  const int32_t* items;
  const int32_t* work_indptr;
  const int32_t* block_table;
  const __nv_bfloat16* q;
  const void* k_scale;
  const void* v_scale;
  __nv_bfloat16* out;
  float* lse;
  __nv_bfloat16* part_o;
  float* part_m;
  float* part_d;
  int32_t* status;
  int64_t q_stride;
  int64_t wait_limit_ns;
  int32_t max_blocks;
  int32_t num_pages;
  int32_t q_heads;
  int32_t kv_heads;
  int32_t group;
  int32_t scale_kind;
  int32_t max_chunks;
  int32_t skip_first_load;
  int32_t q_box_tokens;  // query tokens per TMA box of the item's Q rows (append)
  int32_t softmax_wgs;   // decode: softmax warpgroups in use (1 when every item's rows fit in half)
  float sm_scale_log2;   // sm_scale * log2(e)
  OutEpilogue ep;
  int32_t plain_out;     // expanded rows: no output epilogue, out 32-byte aligned
  const int32_t* cu_seqlens_q;   // device, needed with a tree mask
  const uint8_t* attn_mask;      // [bsz][mask_dim][mask_dim] or null
  int32_t mask_dim;
  int32_t* merge_cnt;    // [total_q][kv_heads] fused-merge counters (decode), or null
  uint64_t* trace;       // [trace_ctas][trace_tiles][16] %globaltimer stamps, or null
  int32_t trace_ctas;
  int32_t trace_tiles;
  int32_t bsz;           // bounds of the work items (checked by the debug build)
  int32_t total_q;
  int32_t num_items;
  int32_t four_bit;      // the items are records of compact slots (item4_from), with
  int32_t part_slots;    // so many slots of partial rows (Plan::part_slots)
};

// One of the products around latent attention (pa_mla_product.cu): x times the weights.
struct MlaProduct {
  int32_t op;              // 0 absorb, 1 project, 2 expand
  int32_t rows, heads;
  const void* x;
  void* out;
  int64_t x_stride, out_stride;
  int32_t* status;
  CUtensorMap tm[4];       // x, weights, output, second output (expand's values)
};

void set_error(const std::string& msg);

// launchers (return a cudaError_t from the launch)
cudaError_t launch_decode(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                          const CUtensorMap& tm_v, cudaStream_t stream);
// decode tiles of at most kWarpDecodeRows packed rows: warp-per-item kernel
cudaError_t launch_decode_warp(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_v, cudaStream_t stream);
cudaError_t launch_append(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                          const CUtensorMap& tm_v, const CUtensorMap& tm_q, cudaStream_t stream);
cudaError_t launch_mla(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_c,
                       cudaStream_t stream);
cudaError_t launch_cache_append(const Plan& plan, const pa_args& a, const void* k_new,
                                const void* v_new, int64_t kv_stride, int32_t* status,
                                cudaStream_t stream);
// the 4-bit cache: attention, quantise-and-write; every cache: read back as bf16
cudaError_t launch_decode4(const Plan& plan, const AttnParams& p, const void* ck, const void* cv,
                           cudaStream_t stream);
cudaError_t launch_decode4_tm(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_k,
                              const void* cv, cudaStream_t stream);
cudaError_t launch_append4(const Plan& plan, const AttnParams& p, const void* ck, const void* cv,
                           const CUtensorMap& tm_q, cudaStream_t stream);
cudaError_t launch_cache_append4(const Plan& plan, const pa_args& a, const void* k_new,
                                 const void* v_new, int64_t kv_stride, int32_t* status,
                                 cudaStream_t stream);
cudaError_t launch_mla_prefill(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_r, const CUtensorMap& tm_v, cudaStream_t stream);
cudaError_t launch_mla_product(const MlaProduct& m, const FaultCfg& fc, cudaStream_t stream);
// expand of many rows, by CTA pairs (its weights' boxes have 128 rows)
cudaError_t launch_mla_expand(const MlaProduct& m, const FaultCfg& fc, int num_sms, cudaStream_t stream);
// queries rotated, K / V rows rotated (K) and written, every cache
cudaError_t launch_rope_append(const Plan& plan, const pa_args& a, const pa_rope& rope, const void* q,
                               int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k_new,
                               const void* v_new, int64_t kv_stride, int32_t* status, cudaStream_t stream);
cudaError_t launch_cache_read(const Plan& plan, const pa_args& a, void* k_out, void* v_out,
                              int64_t kv_stride, int32_t* status, cudaStream_t stream);
cudaError_t launch_merge(const Plan& plan, const WsView& ws, void* out, float* lse,
                         const OutEpilogue& ep, cudaStream_t stream);
cudaError_t launch_gather(const pa_problem& prob, const pa_args& a, int32_t b, int32_t kvh,
                          int32_t pos0, int32_t n, void* dk, void* dv, cudaStream_t stream);

}  // namespace pa
