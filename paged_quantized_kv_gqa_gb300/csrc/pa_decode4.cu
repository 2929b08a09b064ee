// pa_decode4.cu - attention over the 4-bit cache for at most 16 packed query
// rows per (sequence, kv head) tile: decode with small GQA groups.
//
// A warp owns whole work items (sequence, kv head, kv chunk), taken one after
// the other from its CTA's list, and works on half pages of 32 positions:
//   * load: K and V of a half page are one contiguous run of 2304 bytes each
//     (codes and block scales together), so two bulk copies fill a stage of the
//     warp's ring; the warp issues them itself, kStages half pages ahead;
//   * S^T = K Q'^T with mma.sync m16n8k16 (M = 16 positions, N = 8 query rows):
//     lane (g, t) holds dims 32 t .. 32 t + 31 of a position, i.e. 16 bytes of
//     codes and two block scales, and turns each code pair into fp16 with one
//     conversion and one multiplication by its block scale (exact); the dims are
//     dealt to the k steps in whatever order the codes unpack to, Q' following;
//   * running maximum and sum per row in fp32, P = 2^(x - m) in fp16, moved into
//     the B operand by movmatrix;
//   * O^T += V^T P^T: lane (g, t) holds positions 8 t .. 8 t + 7 of 16 dims, a
//     32-bit word of codes each; a 16-dim MMA block is one scale block, so the
//     scale pairs of the positions serve both rows of a lane.
// A piece (a work item) may begin and end inside a page, at a half page.
// Roundings: codes times block scales are exact; P in fp16 (relative error at most 2^-11)
// and the final row.  The mean square error of the outputs is that of the bf16 rounding
// within 3 %; P as two numbers would double the MMAs of PV.  Partial rows are fp32.
// What bounds it: 144 bytes a position and kv head, and per 32 positions about 600
// (FP4) or 690 (int4) warp instructions for 128 code pairs a lane.  Long caches run
// at four fifths of the copy bandwidth, held by the issue slots (two thirds of them
// taken, the rest lost to dependences within four warps a scheduler); short ones by
// what comes before a warp's first half page (item, page ids, copies: about 8 us).
#include <cfloat>

#include "pa_common.cuh"
#include "pa_kv4.cuh"

namespace pa {
namespace {

constexpr int kPage = 64;
constexpr int kRing = 4;               // item records between load and compute cursors
constexpr int kBtStride = 8;           // block-table entries kept per item (512 positions)
constexpr int kScaleBytes = 4096;      // preloaded tensor scales (2 KB each for K and V)
constexpr int kStage4 = 2 * kV4HalfBytes;
constexpr float kTau = 8.0f;           // lazy rescale: P stays below 2^8

template <int NB>
struct D4Cfg {
  // Up to 8 rows: 16 warps of 128 registers, two stages each.  On 8 sequences of
  // 33k-131k positions (64 / 8 heads, FP4) 8, 12, 14 and 16 warps took 188, 164, 173
  // and 157 us, one stage 177, 12 warps of three stages 161; on 24 of up to 3k
  // positions 20.6, 18.0, 19.4 and 17.8 us, one stage 18.0, 12 warps of three 18.3.
  // 9 to 16 rows need twice the accumulators: 8 warps.
  static constexpr int kWarps = decode4_warps(8 * NB);
  static constexpr int kStages = NB == 1 ? 2 : 3;
  static constexpr int kItems = 32;    // CTA item records kept in shared memory
  static constexpr int kScaleOff = kWarps * kStages * kStage4;
  static constexpr int kItemOff = kScaleOff + kScaleBytes;
  static constexpr int kBtOff = kItemOff + kItems * kItemWords * 4;
  static constexpr int kRecOff = kBtOff + kItems * kBtStride * 4;
  static constexpr int kBarOff = kRecOff + kWarps * kRing * 48;
  static constexpr int kMiscOff = kBarOff + kWarps * kStages * 8;
  static constexpr int kQloOff = kMiscOff + 16;        // low parts of Q' (LO = 1, below)
  static constexpr int kBase = kQloOff + 128;          // + alignment slack
  static constexpr int kTotal = kBase + kWarps * NB * 2048;
  static_assert(kTotal <= 232448, "shared memory overflow");
  static_assert(kStages < kRing, "a record outlives its stages");
  // the epilogue stages 8 rows of 128 fp32 at a time in the item's last stage
  static constexpr int kStageRows = 8;
  static_assert(kStageRows * 128 * 4 <= kStage4, "output staging");
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 b16 transpose across the warp
__device__ __forceinline__ uint32_t movtrans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Position (0..31 within the half page) of MMA row g (h = 0) or g + 8 (h = 1)
// of 16-position block b: the positions that lane t's V words unpack to.
template <int FP4>
__device__ __forceinline__ int kpos(int b, int g, int h) {
  return FP4 ? 8 * (g >> 1) + 4 * b + 2 * h + (g & 1) : 8 * (g >> 1) + 2 * b + h + 4 * (g & 1);
}

}  // namespace

// LO > 0: per-channel K scales.  A product of a bf16 query and a bf16 scale has 16
// significant bits; rounded to fp16 it moves a score by up to 2^-11 of sm_scale * sum
// |q k|, and more where it is subnormal (channel scales near 1e-3 and scores near 10: lse
// error 1e-3, as two numbers 5e-6 to 1e-5).  So Q' is the sum of two fp16 numbers there.
// LO = 2, at most 4 rows: the low parts are MMA columns 4 to 7, which have no rows (batch
// of 64 sequences, 4 rows: 45.4 -> 46.4 us; as LO = 1 57.4).  LO = 1: they wait in shared
// memory and go through MMAs of their own (24 sequences, 5 rows: 20.5 -> 23.1 us).
template <int NB, int FP4, bool TREE, int LO>
__global__ void __launch_bounds__(D4Cfg<NB>::kWarps * 32, 1)
    decode4_kernel(const uint8_t* __restrict__ cache_k, const uint8_t* __restrict__ cache_v,
                   const AttnParams p) {
  using C = D4Cfg<NB>;
  constexpr bool PC = LO != 0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int item_begin = p.work_indptr[blockIdx.x];
  const int item_end = p.work_indptr[blockIdx.x + 1];
  const uint64_t limit = (uint64_t)p.wait_limit_ns;
  const int G = p.group;
  const uint32_t g_magic = (65536u + (uint32_t)G - 1u) / (uint32_t)G;   // r / G = (r * g_magic) >> 16 for r < 64
  auto div_g = [&](int r) { return (int)(((uint32_t)r * g_magic) >> 16); };

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff) + warp * C::kStages;
  int32_t* items_s = reinterpret_cast<int32_t*>(smem + C::kItemOff);
  int32_t* bt_s = reinterpret_cast<int32_t*>(smem + C::kBtOff);
  int32_t* rec_ring = reinterpret_cast<int32_t*>(smem + C::kRecOff) + warp * kRing * 12;
  int* next_item = reinterpret_cast<int*>(smem + C::kMiscOff);
  volatile int* abort_any = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  const uint8_t* stage_p = smem + warp * C::kStages * kStage4;
  uint2* qlo = reinterpret_cast<uint2*>(smem + C::kQloOff) + warp * NB * 256 + lane;   // [row block][k step][lane]
  const __nv_bfloat16* ks_s = reinterpret_cast<const __nv_bfloat16*>(smem + C::kScaleOff);
  const __nv_bfloat16* vs_s = ks_s + kScaleBytes / 4;

  const int sc_n = p.scale_kind == PA_SCALE_PER_CHANNEL ? p.kv_heads * kV4Dim
                   : p.scale_kind == PA_SCALE_PER_KV_HEAD ? p.kv_heads : 0;
  const bool sc_smem = sc_n > 0 && sc_n * 2 <= kScaleBytes / 2;
  PA_DEBUG_PROLOGUE(smem, (LO == 1 ? C::kTotal : C::kBase) - 128, p, item_begin, item_end);
  if (threadIdx.x == 0) {
    for (int w = 0; w < C::kWarps; ++w)
      for (int s = 0; s < C::kStages; ++s)
        mbar_init(reinterpret_cast<uint64_t*>(smem + C::kBarOff) + w * C::kStages + s, 1);
    *next_item = item_begin;
    *abort_any = 0;
    fence_mbar_init();
  }
  const int n_staged = min(item_end - item_begin, C::kItems);
  for (int i = threadIdx.x; i < n_staged * kItemWords; i += blockDim.x)
    items_s[i] = p.items[(int64_t)item_begin * kItemWords + i];
  if (sc_smem) {
    __nv_bfloat16* kd = reinterpret_cast<__nv_bfloat16*>(smem + C::kScaleOff);
    __nv_bfloat16* vd = kd + kScaleBytes / 4;
    for (int i = threadIdx.x; i < sc_n; i += blockDim.x) {
      kd[i] = reinterpret_cast<const __nv_bfloat16*>(p.k_scale)[i];
      vd[i] = reinterpret_cast<const __nv_bfloat16*>(p.v_scale)[i];
    }
  }
  __syncthreads();
  // page ids of every staged item of at most kBtStride pages
  for (int idx = threadIdx.x; idx < n_staged * kBtStride; idx += blockDim.x) {
    const int32_t* rec = items_s + (idx / kBtStride) * kItemWords;
    const int k = idx % kBtStride;
    const int pg0 = rec[5] / kPage;
    const int np = (rec[6] + kPage - 1) / kPage - pg0;
    const int nb = p.max_blocks - pg0;
    bt_s[idx] = k < np && k < nb ? p.block_table[(int64_t)rec[0] * p.max_blocks + pg0 + k] : -1;
  }
  __syncthreads();

  // -------------------------------------------------------------- load side
  // warp-uniform cursor over this warp's half pages; the next item is taken
  // when the current one's last half page is issued
  int cur_it = -1, cur_b = 0, cur_kvh = 0, cur_pg0 = 0, cur_nh = 0, cur_h = 0;   // from page cur_pg0 on
  int cur_bt = -1, nxt_bt = -1;       // lane k: page id of page 32 * batch + k of the item
  int pend_it = -1, pend_rec = 0, pend_bt = -1;
  // Q rows of a taken item, read several half pages before they are needed;
  // lane (g, t): dims 32 t .. 32 t + 31 of row 8 j + g
  uint4 qpre[NB][4];
  int qpre_it = -1;
  auto load_q_rows = [&](uint4 (&qr)[NB][4], int tok0, int ntok, int kvh) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int row = LO == 2 ? g & 3 : 8 * j + g;
      const bool valid = row < ntok * G;
      const int tok = valid ? div_g(row) : 0;
      const __nv_bfloat16* src = p.q + (tok0 + tok) * p.q_stride + (kvh * G + (valid ? row - tok * G : 0)) * kV4Dim +
                                 32 * t;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        qr[j][k] = make_uint4(0, 0, 0, 0);
        if (valid) qr[j][k] = __ldg(reinterpret_cast<const uint4*>(src) + k);
      }
    }
  };
  uint32_t n_load = 0;                // half pages issued by this warp
  int st_load = 0;                    // the stage of the next one
  uint32_t k_load = 0;                // items started on the load side
  const bool skip_hook = p.skip_first_load && blockIdx.x == 0;   // failure-detection test hook
  uint32_t skipped_n = 0xFFFFFFFFu;

  auto bt_at = [&](int b, int pg0, int pg) -> int {
    return pg < p.max_blocks - pg0 ? p.block_table[(int64_t)b * p.max_blocks + pg0 + pg] : -1;
  };
  auto take_pending = [&]() {
    int it = 0;
    if (lane == 0) it = atomicAdd(next_item, 1);
    it = __shfl_sync(0xffffffffu, it, 0);
    pend_it = it < item_end ? it : -1;
    if (pend_it >= 0) {
      const int k = pend_it - item_begin;
      if (lane < kItemWords)
        pend_rec = k < n_staged ? items_s[k * kItemWords + lane] : p.items[(int64_t)pend_it * kItemWords + lane];
      const int b = __shfl_sync(0xffffffffu, pend_rec, 0);
      const int pg0 = __shfl_sync(0xffffffffu, pend_rec, 5) / kPage;
      const int kv1 = __shfl_sync(0xffffffffu, pend_rec, 6);
      const int np = (kv1 + kPage - 1) / kPage - pg0;
      if (k < n_staged && np <= kBtStride) pend_bt = lane < np ? bt_s[k * kBtStride + lane] : -1;
      else pend_bt = lane < np ? bt_at(b, pg0, lane) : -1;
      if (qpre_it < 0) {   // the previous prefetch has been used
        load_q_rows(qpre, __shfl_sync(0xffffffffu, pend_rec, 2), __shfl_sync(0xffffffffu, pend_rec, 3) & 0xFFFF,
                    __shfl_sync(0xffffffffu, pend_rec, 1));
        qpre_it = pend_it;
      }
    }
  };
  // issues the next half page of this warp's sequence
  auto issue_next = [&]() -> bool {
    bool skip_copy = false;
    if (cur_it < 0 || cur_h == cur_nh) {
      if (pend_it < 0) return false;
      cur_it = pend_it;
      cur_b = __shfl_sync(0xffffffffu, pend_rec, 0);
      cur_kvh = __shfl_sync(0xffffffffu, pend_rec, 1);
      const int kv0 = __shfl_sync(0xffffffffu, pend_rec, 5);
      const int kv1 = __shfl_sync(0xffffffffu, pend_rec, 6);
      cur_pg0 = kv0 / kPage;
      cur_nh = (kv1 + kV4Half - 1) / kV4Half - 2 * cur_pg0;
      cur_h = kv0 / kV4Half - 2 * cur_pg0;   // a piece may begin with a second half
      cur_bt = pend_bt;
      nxt_bt = (lane + 32) * 2 < cur_nh ? bt_at(cur_b, cur_pg0, 32 + lane) : -1;
      int32_t* slot = rec_ring + (k_load % kRing) * 12;   // the record for the compute side
      if (lane < kItemWords) slot[lane] = pend_rec;
      if (lane == kItemWords) slot[kItemWords] = cur_it;
      __syncwarp();
      ++k_load;
      skip_copy = skip_hook && cur_it == item_begin;
      pend_it = -1;
    } else if ((cur_h & 63) == 0) {
      cur_bt = nxt_bt;
      const int pg = (cur_h >> 1) + 32 + lane;
      nxt_bt = pg * 2 < cur_nh ? bt_at(cur_b, cur_pg0, pg) : -1;
    }
    const int page = __shfl_sync(0xffffffffu, cur_bt, (cur_h >> 1) & 31);
    if (lane == 0 && !skip_copy) {
      uint64_t* bar = &full[st_load];
      fence_proxy_async_smem();   // this stage's earlier reads before the new writes
      mbar_arrive_expect_tx(bar, (uint32_t)kStage4);
      const bool ok = page >= 0 && page < p.num_pages;
      if (!ok) record_status(p.status, PA_ERR_BAD_PAGE, cur_it);
      // a bad page id reads page 0 instead (the run's status says so)
      const int64_t off = (int64_t)((ok ? page : 0) * p.kv_heads + cur_kvh) * kV4Slab + (cur_h & 1) * kV4HalfBytes;
      uint8_t* st = smem + (warp * C::kStages + st_load) * kStage4;
      bulk_load(st, cache_k + off, kV4HalfBytes, bar);
      bulk_load(st + kV4HalfBytes, cache_v + off, kV4HalfBytes, bar);
    }
    __syncwarp();
    if (skip_copy) skipped_n = n_load;
    ++cur_h;
    ++n_load;
    if (++st_load == C::kStages) st_load = 0;
    if (cur_h == cur_nh) take_pending();   // the next item, one stage ahead of its use
    return true;
  };

  // ------------------------------------------------------------ compute side
  bool fail = false;
  take_pending();
  for (int s = 0; s < C::kStages; ++s)
    if (!issue_next()) break;

  uint32_t n_comp = 0, k_comp = 0;
  int st_comp = 0;
  uint32_t ph_comp = 0;
  while (!fail && n_comp < n_load) {
    const int32_t* slot = rec_ring + (k_comp % kRing) * 12;
    const Item m = item4_from<kV4Half>(*reinterpret_cast<const int4*>(slot), *reinterpret_cast<const int4*>(slot + 4));
    const int it = slot[kItemWords];
    const int n_rows = m.ntok * G;
    const int nh = m.ntiles;   // half pages
    float c_log2 = p.sm_scale_log2 * kFold8<FP4>;
    if (p.scale_kind == PA_SCALE_GLOBAL) c_log2 *= reinterpret_cast<const float*>(p.k_scale)[0];
    else if (p.scale_kind == PA_SCALE_PER_KV_HEAD)
      c_log2 *= __bfloat162float(sc_smem ? ks_s[m.kvh] : reinterpret_cast<const __nv_bfloat16*>(p.k_scale)[m.kvh]);
    // a sign goes into Q'; a scale of 0 becomes one too small to matter (-inf * 0 is NaN)
    const float c_abs = fmaxf(fabsf(c_log2), 1e-30f), sgn = c_log2 < 0.f ? -1.f : 1.f;
    const float c_inv = __fdividef(1.f, c_abs);
    int tok0_local = 0, pre_len = 0;
    const uint8_t* tmask = nullptr;
    if constexpr (TREE) {
      tok0_local = m.tok0 - p.cu_seqlens_q[m.b];
      pre_len = m.cbase - tok0_local;
      tmask = p.attn_mask + (int64_t)m.b * p.mask_dim * p.mask_dim;
    }

    // Q' fragments of row 8 j + g: k step ks takes dims 32 t + 8 (ks / 2) + the
    // pairs that the codes of that word unpack to
    uint32_t qf[NB][8][2];
    {
      uint4 qr[NB][4];
      if (it == qpre_it) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) qr[j][k] = qpre[j][k];
        qpre_it = -1;
      } else {
        load_q_rows(qr, m.tok0, m.ntok, m.kvh);
      }
      const __nv_bfloat16* sk = (sc_smem ? ks_s : reinterpret_cast<const __nv_bfloat16*>(p.k_scale)) +
                                (PC ? m.kvh * kV4Dim + 32 * t : 0);
      const bool sk16 = PC && (reinterpret_cast<uintptr_t>(sk) & 15) == 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float sc[8];
        if (sk16) {
          const uint4 u = *reinterpret_cast<const uint4*>(sk + 8 * w);
          const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[2 * e] = __uint_as_float(x[e] << 16) * sgn;
            sc[2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u) * sgn;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) sc[e] = PC ? __bfloat162float(sk[8 * w + e]) * sgn : sgn;
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const uint32_t u[4] = {qr[j][w].x, qr[j][w].y, qr[j][w].z, qr[j][w].w};
          float f[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b2 = *reinterpret_cast<const __nv_bfloat162*>(&u[e]);
            f[2 * e] = __low2float(b2) * sc[2 * e];
            f[2 * e + 1] = __high2float(b2) * sc[2 * e + 1];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e0 = FP4 ? 2 * i : i, e1 = FP4 ? 2 * i + 1 : i + 4;
            const uint32_t hi = pack_half2(f[e0], f[e1]);
            qf[j][2 * w + (i >> 1)][i & 1] = hi;
            if constexpr (LO == 2) {
              const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              if (g >= 4) qf[j][2 * w + (i >> 1)][i & 1] = pack_half2(f[e0] - h.x, f[e1] - h.y);
            }
            if constexpr (LO == 1) {
              const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              reinterpret_cast<uint32_t*>(qlo + (8 * j + 2 * w + (i >> 1)) * 32)[i & 1] =
                  pack_half2(f[e0] - h.x, f[e1] - h.y);
            }
          }
        }
      }
    }

    float o[NB][8][4];
    float mrow[NB][2], mlim[NB][2], lrow[NB][2];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
#pragma unroll
      for (int d = 0; d < 8; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][d][e] = 0.f;
      mrow[j][0] = mrow[j][1] = mlim[j][0] = mlim[j][1] = -INFINITY;
      lrow[j][0] = lrow[j][1] = 0.f;
    }

    for (int hp = 0; hp < nh; ++hp) {
      if (!wait_or_abort(&full[st_comp], ph_comp, limit, abort_any, 32)) {
        if (!*abort_any) record_status(p.status, PA_ERR_DEVICE_TIMEOUT, it);
        *abort_any = 1;
        fail = true;
        break;
      }
      if (lane == 0 && warp < 4) trace_ev(p, n_comp, 12 + warp);
      const uint8_t* kst = stage_p + st_comp * kStage4;
      const uint8_t* vst = kst + kV4HalfBytes;
      const int pos0 = m.kv0 + hp * kV4Half;

      // ---- S^T = K Q'^T for the two 16-position blocks
      float s[2][NB][4];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[b][j][e] = 0.f;
        float sl[NB][4] = {};   // the low parts' sums, a chain of their own
        uint4 kr[2];
        uint32_t ksc[2][2], koff[2][2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = kpos<FP4>(b, g, h);
          kr[h] = *reinterpret_cast<const uint4*>(kst + r * (kV4Dim / 2) + 16 * t);
          scale_pair_fold8<FP4>(*reinterpret_cast<const uint16_t*>(kst + kV4Codes + r * kV4Nblk + 2 * t), ksc[h],
                                koff[h]);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a[4], c[4];
          codes8<FP4>(word_of(kr[0], w), a);
          codes8<FP4>(word_of(kr[1], w), c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = scaled_fold8<FP4>(a[i], ksc[0][w >> 1], koff[0][w >> 1][i & 1]);
            c[i] = scaled_fold8<FP4>(c[i], ksc[1][w >> 1], koff[1][w >> 1][i & 1]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              mma_16816(s[b][j], a[2 * i], c[2 * i], a[2 * i + 1], c[2 * i + 1], qf[j][2 * w + i][0],
                        qf[j][2 * w + i][1]);
              if constexpr (LO == 1) {
                const uint2 lo = qlo[(8 * j + 2 * w + i) * 32];
                mma_16816(sl[j], a[2 * i], c[2 * i], a[2 * i + 1], c[2 * i + 1], lo.x, lo.y);
              }
            }
        }
        if constexpr (LO == 1) {
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[b][j][e] += sl[j][e];
        }
        if constexpr (LO == 2) {   // (columns 4 to 7 end up as copies of 0 to 3, not stored)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[b][0][e] += __shfl_xor_sync(0xffffffffu, s[b][0][e], 2);
        }
      }

      uint16_t* vs16 = reinterpret_cast<uint16_t*>(smem + (warp * C::kStages + st_comp) * kStage4);   // [8][32]
      // V scales as fp16, once per half page, over the K codes (every lane has read
      // its own): lane (g, t) converts block g's positions 8t .. 8t+7, stored in the
      // order their codes unpack to (int4: a plane of offsets behind the scales).
      // Positions past the chunk's end get scale 0: their bytes may hold
      // anything, and a code is finite whatever it is.
      {
        uint2 sw = *reinterpret_cast<const uint2*>(vst + kV4Codes + g * kV4Half + 8 * t);
        const int left = m.kv1 - pos0 - 8 * t;   // valid positions of these eight
        keep_scales(sw, left);
        uint32_t f[4];
        scales8<FP4>(sw, f);
        if constexpr (!FP4) {
          uint32_t e0, e2, unused;
          fold8(f[0], f[0], e0, unused);
          fold8(f[2], f[2], e2, unused);
          uint32_t o1, o3;
          fold8(f[1], f[1], unused, o1);
          fold8(f[3], f[3], unused, o3);
          __syncwarp();
          *reinterpret_cast<uint4*>(vs16 + kV4Nblk * kV4Half + g * kV4Half + 8 * t) = make_uint4(e0, o1, e2, o3);
        } else {
          __syncwarp();
        }
        *reinterpret_cast<uint4*>(vs16 + g * kV4Half + 8 * t) = make_uint4(f[0], f[1], f[2], f[3]);
      }

      // ---- mask, running max, P (scores stay unscaled; the scale is in the exponent)
      const bool need_mask = (pos0 + kV4Half > m.kv1) || (pos0 + kV4Half - 1 > m.cbase) ||
                             (TREE && pos0 + kV4Half > pre_len);
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int jpos = pos0 + kpos<FP4>(b, g, h);
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (need_mask) {
                const int r = 8 * j + 2 * t + e;
                bool vis = jpos < m.kv1 && jpos <= m.cbase + div_g(r);
                if (TREE && vis && jpos >= pre_len && r < n_rows) {
                  const int tl = tok0_local + div_g(r);
                  vis = tmask[tl * p.mask_dim + (jpos - pre_len)] != 0;
                }
                s[b][j][2 * h + e] = vis ? s[b][j][2 * h + e] : -INFINITY;
              }
            }
        }
      // The running maximum moves only when some score exceeds it by 2^kTau (the
      // vote makes that one decision for the warp); P and the sums stay relative
      // to it in fp32.
      bool exceed = false;
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          exceed |= fmaxf(fmaxf(s[0][j][e], s[0][j][2 + e]), fmaxf(s[1][j][e], s[1][j][2 + e])) > mlim[j][e];
      if (__any_sync(0xffffffffu, exceed)) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = fmaxf(fmaxf(s[0][j][e], s[0][j][2 + e]), fmaxf(s[1][j][e], s[1][j][2 + e]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float mo = mrow[j][e], mn = fmaxf(mo, v * c_abs);
            // a row without a visible position so far keeps mrow = -inf, O = 0
            const float al = mo == -INFINITY ? 0.f : fast_exp2(mo - mn);
            mrow[j][e] = mn;
            mlim[j][e] = mn == -INFINITY ? -INFINITY : (mn + kTau) * c_inv;
            lrow[j][e] *= al;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              o[j][d][e] *= al;
              o[j][d][2 + e] *= al;
            }
          }
      }
      uint32_t pb[2][NB][2];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const float mu0 = mrow[j][0] == -INFINITY ? 0.f : mrow[j][0];
        const float mu1 = mrow[j][1] == -INFINITY ? 0.f : mrow[j][1];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float p0 = fast_exp2(fmaf(s[b][j][0], c_abs, -mu0));
          const float p1 = fast_exp2(fmaf(s[b][j][1], c_abs, -mu1));
          const float p2 = fast_exp2(fmaf(s[b][j][2], c_abs, -mu0));
          const float p3 = fast_exp2(fmaf(s[b][j][3], c_abs, -mu1));
          lrow[j][0] += p0 + p2;
          lrow[j][1] += p1 + p3;
          pb[b][j][0] = movtrans(pack_half2(p0, p1));
          pb[b][j][1] = movtrans(pack_half2(p2, p3));
        }
      }

      // ---- O^T += V^T P^T
      __syncwarp();   // the fp16 scales of every lane are in place
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        uint32_t a[4], c[4];
        codes8<FP4>(*reinterpret_cast<const uint32_t*>(vst + (16 * d + g) * (kV4Half / 2) + 4 * t), a);
        codes8<FP4>(*reinterpret_cast<const uint32_t*>(vst + (16 * d + g + 8) * (kV4Half / 2) + 4 * t), c);
        const uint4 sv = *reinterpret_cast<const uint4*>(vs16 + d * kV4Half + 8 * t);
        uint4 nv = sv;
        if constexpr (!FP4) nv = *reinterpret_cast<const uint4*>(vs16 + kV4Nblk * kV4Half + d * kV4Half + 8 * t);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t x[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x[2 * i] = scaled_fold8<FP4>(a[2 * b + i], word_of(sv, 2 * b + i), word_of(nv, 2 * b + i));
            x[2 * i + 1] = scaled_fold8<FP4>(c[2 * b + i], word_of(sv, 2 * b + i), word_of(nv, 2 * b + i));
          }
#pragma unroll
          for (int j = 0; j < NB; ++j) mma_16816(o[j][d], x[0], x[1], x[2], x[3], pb[b][j][0], pb[b][j][1]);
        }
      }

      // the stage is free (the epilogue uses the item's last one)
      __syncwarp();
      if (lane == 0 && warp < 12) trace_ev(p, n_comp, warp);
      ++n_comp;
      if (++st_comp == C::kStages) {
        st_comp = 0;
        ph_comp ^= 1;
      }
      if (hp + 1 < nh) issue_next();
    }
    if (fail) break;

    // ---- epilogue.  Partial rows leave as they sit in the accumulators: a store
    // of the warp writes eight consecutive dims of four rows, whole 32-byte
    // sectors of fp32.  Final rows (bf16 or int8) go 8 at a time through the
    // item's last stage as fp32 [8 rows][128 dims] (dims of row r XOR
    // 8 ((r >> 1) & 3): no bank conflicts) and leave as 16-byte pieces.
    const bool final_row = m.nch == 1;
    const bool per_channel = p.scale_kind == PA_SCALE_PER_CHANNEL;
    const float vs_head = kFold8<FP4> * (p.scale_kind == PA_SCALE_GLOBAL ? reinterpret_cast<const float*>(p.v_scale)[0]
                          : p.scale_kind == PA_SCALE_PER_KV_HEAD
                              ? __bfloat162float(sc_smem ? vs_s[m.kvh]
                                                         : reinterpret_cast<const __nv_bfloat16*>(p.v_scale)[m.kvh])
                              : 1.f);
    const __nv_bfloat16* vsc = (sc_smem ? vs_s : reinterpret_cast<const __nv_bfloat16*>(p.v_scale)) +
                               (per_channel ? m.kvh * kV4Dim : 0);
    float inv[NB][2];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = lrow[j][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        inv[j][e] = l > 0.f ? __frcp_rn(l) * vs_head : 0.f;
        const int r = 8 * j + 2 * t + e;
        if (g == 0 && r < n_rows) {
          const int dt = div_g(r);
          const int token = m.tok0 + dt;
          const int head = m.kvh * G + r - dt * G;
          const float ln2 = 0.69314718055994530942f;
          const float mr = mrow[j][e];
          if (final_row) {
            if (p.lse != nullptr)
              p.lse[(int64_t)token * p.q_heads + head] = l > 0.f ? (mr + __log2f(l)) * ln2 : -INFINITY;
          } else {
            const int64_t sp = (int64_t)(m.chunk + dt * m.nch) * p.q_heads + head;
            p.part_m[sp] = l > 0.f ? mr * ln2 : -INFINITY;
            p.part_d[sp] = l;
          }
        }
      }
    if (!final_row) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * j + 2 * t + e;
          if (r < n_rows) {
            const int dt = div_g(r);
            float* dst = reinterpret_cast<float*>(p.part_o) +
                         ((int64_t)(m.chunk + dt * m.nch) * p.q_heads + m.kvh * G + r - dt * G) *
                             kV4Dim + g;
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float v = o[j][d][2 * h + e] * inv[j][e];
                if (per_channel) v *= __bfloat162float(vsc[16 * d + 8 * h + g]);
                dst[16 * d + 8 * h] = v;
              }
          }
        }
    } else {
      const bool plain = p.ep.shift == nullptr && p.ep.smooth == nullptr && !p.ep.int8_out;
      float* stg = reinterpret_cast<float*>(smem + (warp * C::kStages + (st_comp == 0 ? C::kStages : st_comp) - 1) * kStage4);
      const bool vec = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              stg[(2 * t + e) * kV4Dim + ((16 * d + g + 8 * h) ^ (8 * t))] = o[j][d][2 * h + e] * inv[j][e];
        __syncwarp();
#pragma unroll 1
        for (int idx = lane; idx < min(8, n_rows - 8 * j) * 16; idx += 32) {
          const int rr = idx >> 4, c = idx & 15;   // row 8 j + rr, dims 8c .. 8c+7
          const float* src = stg + rr * kV4Dim + ((8 * c) ^ (8 * ((rr >> 1) & 3)));
          const float4 a = *reinterpret_cast<const float4*>(src);
          const float4 b = *reinterpret_cast<const float4*>(src + 4);
          float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          if (per_channel) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= __bfloat162float(vsc[8 * c + k]);
          }
          const int dt = div_g(8 * j + rr);
          const int token = m.tok0 + dt;
          const int head = m.kvh * G + 8 * j + rr - dt * G;
          const int64_t oi = ((int64_t)token * p.q_heads + head) * kV4Dim + 8 * c;
          if (plain && vec) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
              w[k] = *reinterpret_cast<uint32_t*>(&b2);
            }
            *reinterpret_cast<uint4*>(p.out + oi) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
            ep_store8(p.ep, p.out, oi, head * kV4Dim + 8 * c, v, vec);
          }
        }
        __syncwarp();   // the staged rows are read before they are overwritten
      }
    }
    ++k_comp;
    issue_next();   // the stage of the item's last half page
  }

  if (fail || *abort_any) {
    if (!*abort_any) *abort_any = 1;
    // every copy this warp issued lands before the CTA's shared memory is released
    if (lane == 0)
      for (uint32_t n = n_comp; n < n_load; ++n)
        if (n != skipped_n) mbar_wait(&full[n % C::kStages], (n / C::kStages) & 1, kDrainNs);
    __syncwarp();
  }
  pdl_launch_dependents();   // the merge grid may be scheduled while the last CTAs finish
}

template <int NB, int FP4, int LO>
static cudaError_t launch_d4(const Plan& plan, const AttnParams& p, const uint8_t* ck, const uint8_t* cv,
                             cudaStream_t stream) {
  auto kern = p.attn_mask != nullptr ? decode4_kernel<NB, FP4, true, LO> : decode4_kernel<NB, FP4, false, LO>;
  const int smem = LO == 1 ? D4Cfg<NB>::kTotal : D4Cfg<NB>::kBase;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<plan.num_ctas, D4Cfg<NB>::kWarps * 32, smem, stream>>>(ck, cv, p);
  return cudaGetLastError();
}

cudaError_t launch_decode4(const Plan& plan, const AttnParams& p, const void* ck, const void* cv,
                           cudaStream_t stream) {
  const bool fp4 = plan.prob.kv_dtype == PA_KV_FP4_E2M1;
  const uint8_t* k = static_cast<const uint8_t*>(ck);
  const uint8_t* v = static_cast<const uint8_t*>(cv);
  const int rows = plan.max_q * (plan.prob.q_heads / plan.prob.kv_heads);
  const bool pc = plan.prob.scale_kind == PA_SCALE_PER_CHANNEL;
  if (rows > 16) return cudaErrorInvalidValue;
  auto launch = rows <= 8 ? (!pc ? (fp4 ? launch_d4<1, 1, 0> : launch_d4<1, 0, 0>)
                             : rows <= 4 ? (fp4 ? launch_d4<1, 1, 2> : launch_d4<1, 0, 2>)
                                         : (fp4 ? launch_d4<1, 1, 1> : launch_d4<1, 0, 1>))
                          : (pc ? (fp4 ? launch_d4<2, 1, 1> : launch_d4<2, 0, 1>)
                                : (fp4 ? launch_d4<2, 1, 0> : launch_d4<2, 0, 0>));
  return launch(plan, p, k, v, stream);
}

}  // namespace pa
