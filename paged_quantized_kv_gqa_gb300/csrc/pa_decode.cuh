// pa_decode.cuh - the tensor-memory decode kernel of the 4-bit cache: 17 to 64 packed
// query rows (decode and speculative verify), tcgen05 + TMA, sm_103a.
//
// The method is pa_decode.cu's (swap-AB: 128 KV positions on the TMEM lanes, the packed
// rows as the MMA's N; S^T = K Q'^T, O^T += V^T P^T; softmax warpgroups of half of the
// rows each; K, V and S double-buffered, P^T four-deep, Q' and O per item).  What
// differs, and why the two are separate sources (one template for both moved the 8-bit
// kernel's register allocation: 1.52 -> 1.56 to 1.65 ms on spec-verify-4):
//   * a page's K slab arrives as a 72-row box of 64 bytes with 64B swizzle (a thread
//     reads one position's 64 code bytes: without the swizzle eight neighbours would
//     share banks), its V slab by a bulk copy (a thread reads 16 bytes of its dim);
//   * 640 threads: a converter warpgroup each for K and V, which multiply code pairs by
//     their block scales (exact in fp16; int4 K with the code offset and 1/8 in the
//     same instruction, 307.1 -> 303.1 us on 48 rows; doing V so too needs a second
//     read of scales per word: 305.2); V's scales are converted once per warp and read
//     back as fp16.  S and PV are issued by a warp each that sleeps on its barriers;
//   * int4 codes unpack in the order 0 4 1 5 2 6 3 7 of each eight: the dims of Q' take
//     the same order, and a P^T row is written at its position's place in that order;
//   * partial rows are fp32, merged by the separate kernel only; P is fp16 as there (it
//     adds about 3 % to the mean square error of the rows' bf16 rounding);
//   * per-channel K scales go into Q': the product of a bf16 query and a bf16 scale has
//     16 significant bits and is the sum of two fp16 numbers, as in the warp kernel, with
//     eight more MMAs a tile for the low parts (PC; 48 rows, int4: 301 -> 322 us, FP4
//     278 -> 294).  As one number a score moves by up to 2^-11 of its terms' magnitude:
//     with channel scales near 1e-3 and scores near 10 the lse moved by 2e-3 (now 1e-5).
//
// Included by pa_decode4_tm.cu.
#pragma once

#include <cfloat>

#include "pa_common.cuh"
#include "pa_decode_tile.cuh"
#include "pa_kv4.cuh"

namespace pa {
namespace {

constexpr int kSlot4 = 5120;                     // a slab's place in a stage (64B-swizzled boxes
                                                 // start on 512 bytes)
constexpr int kVOff = 2 * kSlot4;                // V slabs behind the two K slabs
constexpr int kStageBytes = 4 * kSlot4;          // K (2 pages) + V (2 pages)
constexpr int kVs16Warp = 2 * kTileTok * 2;      // a V converter warp's scales as fp16 [2 blocks][128]
static_assert(kSlot4 >= kV4Slab && kSlot4 % 512 == 0, "stage layout");
// Warpgroups: two softmax, a converter for K and one for V (a code needs more steps
// than a byte, and one group for both held the pipeline up), and IO, whose warps copy
// and issue S and PV from a warp each.  (A softmax warpgroup for every 16 rows
// instead of two for all measured slower, 334 against 319 us on 48 rows.)
constexpr int kThreads = 640;
constexpr int kWarpTma = 16;
constexpr int kWarpS = 17;                       // issues S, the next warp PV

template <int NR>
struct Smem {
  static constexpr int kStages = kPageStages;
  static constexpr int kQ = kStages * kStageBytes;         // Q'[2]
  static constexpr int kQlo = kQ + 2 * NR * 256;           // its low parts [2] (per-channel K scales)
  static constexpr int kP = kQlo + 2 * NR * 256;           // P^T ring
  static constexpr int kRed = kP + kPBufs * kPBufBytes;    // [4][NR] warp maxima
  static constexpr int kRedL = kRed + 4 * NR * 4;          // [4][NR] warp row sums
  static constexpr int kLsum = kRedL + 4 * NR * 4;         // [2][NR] 1/l per item (by parity)
  static constexpr int kM = kLsum + 2 * NR * 4;            // [NR] running max
  static constexpr int kAlpha = kM + NR * 4;               // [NR] rescale factors
  static constexpr int kBars = kAlpha + NR * 4;
  // full[S], empty[S], kready[2], sfull[2], sfree[2], pready[4], vready[2], pvdone[4]
  static constexpr int kNumBars = 2 * kStages + 2 + 2 + 2 + kPBufs + 2 + kPBufs;
  static constexpr int kMisc = kBars + kNumBars * 8;       // tmem addr, abort flags
  static constexpr int kItems = kMisc + 32;                // [kCachedItems][8] int32
  static constexpr int kScales = kItems + kCachedItems * kItemWords * 4;   // k, v [kCachedHeads] fp32
  static constexpr int kVs16 = kScales + 2 * kCachedHeads * 4;             // [4 warps] V scales
  static constexpr int kTotal = kVs16 + 4 * kVs16Warp + 1024;              // + alignment slack
  static_assert(kVs16 % 16 == 0, "the scales are read as 16-byte vectors");
  static_assert(kItems % 16 == 0, "item records are read as int4");
  static_assert(kQ % 1024 == 0 && kQlo % 1024 == 0 && kP % 1024 == 0, "swizzled operands start on 1 KB");
  static_assert(kTotal <= 232448, "shared memory overflow");
};

}  // namespace

// KV: PA_KV_*; PC: per-channel K scales; cv: the V cache
template <int NR, int KV, bool TREE, bool PC>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tm_k, const uint8_t* __restrict__ cv, const AttnParams p) {
  constexpr int FP4 = KV == PA_KV_FP4_E2M1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  using SM = Smem<NR>;
  using TM = Tm<NR>;
  constexpr int kStages = SM::kStages;
  constexpr int NH = NR / 2;       // rows per softmax warpgroup
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::kBars);
  uint64_t* full = bars;
  uint64_t* empty = full + kStages;
  uint64_t* kready = empty + kStages;
  uint64_t* sfull = kready + 2;
  uint64_t* sfree = sfull + 2;
  uint64_t* pready = sfree + 2;
  uint64_t* vready = pready + kPBufs;
  uint64_t* pvdone = vready + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kMisc);
  volatile int* abort_any = reinterpret_cast<volatile int*>(smem + SM::kMisc + 4);
  volatile int* abort_grp = reinterpret_cast<volatile int*>(smem + SM::kMisc + 8);  // [2]
  float* red = reinterpret_cast<float*>(smem + SM::kRed);
  float* red_l = reinterpret_cast<float*>(smem + SM::kRedL);
  float* lsum_s = reinterpret_cast<float*>(smem + SM::kLsum);
  float* m_s = reinterpret_cast<float*>(smem + SM::kM);
  float* alpha_s = reinterpret_cast<float*>(smem + SM::kAlpha);
  const uint32_t s_base = smem_u32(smem);
  const uint32_t q_s = s_base + SM::kQ;
  const uint32_t p_s = s_base + SM::kP;

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int wg = warp >> 2;         // warpgroup: 0, 1 softmax; 2, 3 converters of K, V; 4 IO
  const int item_begin = p.work_indptr[blockIdx.x];
  const int item_end = p.work_indptr[blockIdx.x + 1];
  const uint64_t limit = (uint64_t)p.wait_limit_ns;
  const int G = p.group;
  PA_DEBUG_PROLOGUE(smem, (SM::kTotal) - 1024, p, item_begin, item_end);

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 8);   // the warps that read a stage
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(&kready[j], 4);
      mbar_init(&sfull[j], 1);
      mbar_init(&sfree[j], 4 * p.softmax_wgs);
      mbar_init(&vready[j], 4);
    }
    for (int j = 0; j < kPBufs; ++j) {
      mbar_init(&pready[j], 4 * p.softmax_wgs);
      mbar_init(&pvdone[j], 1);
    }
    *abort_any = 0;
    abort_grp[0] = 0;
    abort_grp[1] = 0;
    fence_mbar_init();
  }
  int32_t* items_s = reinterpret_cast<int32_t*>(smem + SM::kItems);
  float* ks_s = reinterpret_cast<float*>(smem + SM::kScales);
  float* vs_s = ks_s + kCachedHeads;
  const ItemSrc<true> isrc{items_s, p.items, item_begin, min(item_end - item_begin, kCachedItems)};
  for (int i = tid; i < isrc.n_cached * kItemWords; i += kThreads)
    items_s[i] = p.items[(int64_t)item_begin * kItemWords + i];
  // per-kv-head or global scales (per-channel ones are read per item)
  const bool sc_cached = p.scale_kind != PA_SCALE_PER_CHANNEL && p.kv_heads <= kCachedHeads;
  if (sc_cached)
    for (int h = tid; h < p.kv_heads; h += kThreads) {
      ks_s[h] = load_scale(p.k_scale, p.scale_kind, h);
      vs_s[h] = load_scale(p.v_scale, p.scale_kind, h);
    }
  auto kscale = [&](int kvh) { return sc_cached ? ks_s[kvh] : load_scale(p.k_scale, p.scale_kind, kvh); };
  auto vscale = [&](int kvh) { return sc_cached ? vs_s[kvh] : load_scale(p.v_scale, p.scale_kind, kvh); };
  if (warp == 0) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PA_DEBUG_POISON_TMEM(tmem, kTmemCols, warp);
  // this warp's TMEM lane quarter (a warp may only touch lanes 32*(warp%4) ..)
  const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);

  if (warp == kWarpTma) {
    // ================================================================ TMA
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      uint32_t g = 0;
      int issued_g[kStages];
      for (int s = 0; s < kStages; ++s) issued_g[s] = -1;
      bool ok = true;
      for (int it = item_begin; it < item_end && ok; ++it) {
        const Item m = isrc.at(it);
        const int32_t* bt = p.block_table + (int64_t)m.b * p.max_blocks;
        for (int t = 0; t < m.ntiles; ++t, ++g) {
          const int stage = g % kStages;
          const uint32_t ph = (g / kStages) & 1;
          const int pos0 = m.kv0 + t * kTileTok;
          const int npg = (m.kv1 - pos0) > kPage ? 2 : 1;
          // the page ids are read before waiting so their latency overlaps the wait
          int pages[2];
          pages[0] = bt[pos0 / kPage];
          pages[1] = npg == 2 ? bt[pos0 / kPage + 1] : 0;
          if (!dwait(&empty[stage], ph ^ 1, limit, abort_any)) {
            if (!*abort_any) record_status(p.status, PA_ERR_DEVICE_TIMEOUT, it);
            *abort_any = 1;
            ok = false;
            break;
          }
          if (p.skip_first_load && g == 0) continue;  // failure-detection test hook
          mbar_arrive_expect_tx(&full[stage], (uint32_t)(npg * 2 * kV4Slab));
          issued_g[stage] = (int)g;
          uint8_t* st = smem + stage * kStageBytes;
          for (int pg = 0; pg < npg; ++pg) {
            const int page = pages[pg];
            const bool in_pool = page >= 0 && page < p.num_pages;
            if (!in_pool) record_status(p.status, PA_ERR_BAD_PAGE, it);   // reads page 0 instead
            const int slab = (in_pool ? page : 0) * p.kv_heads + m.kvh;
            tma_load_2d(st + pg * kSlot4, &tm_k, &full[stage], 0, slab * (kV4Slab / 64));
            bulk_load(st + kVOff + pg * kSlot4, cv + (int64_t)slab * kV4Slab, kV4Slab, &full[stage]);
          }
          trace_ev(p, g, 0);
        }
      }
      for (int s = 0; s < kStages; ++s)   // every issued load lands before exit
        if (issued_g[s] >= 0) mbar_wait(&full[s], ((uint32_t)issued_g[s] / kStages) & 1, kDrainNs);
    }
  } else if (warp == kWarpS || warp == kWarpS + 1) {
    // ================================================================ MMA issue
    // S and PV each have a warp that sleeps on its barriers: one warp polling both
    // queues took issue slots from the converters on its sub-partition
    const bool is_s = warp == kWarpS;
    auto mwait = [&](uint64_t* bar, uint32_t parity) { return wait_or_abort(bar, parity, limit, abort_any, 100); };
    const uint32_t idesc = is_s ? idesc_f16_f32(128, NR) : idesc_f16_f32_bmn(128, NR);
    TileCursor<true> c;
    c.init(isrc, item_begin, item_end);
    uint32_t g = 0, commits[kPBufs] = {0, 0, 0, 0};
    bool ok = true;
    for (; c.valid(); c.advance(), ++g) {
      if (is_s) {
        if (!mwait(&kready[g & 1], (g >> 1) & 1) ||
            (g >= 2 && !mwait(&sfree[g & 1], ((g - 2) >> 1) & 1))) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t qb = q_s + ((c.it - item_begin) & 1) * NR * 256;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tmem + TM::S0 + (g & 1) * NR, tmem + TM::K0 + (g & 1) * 64 + 8 * kk,
                   sdesc_k128(qb + (kk >> 2) * NR * 128 + (kk & 3) * 32), idesc, kk > 0 ? 1u : 0u);
          if constexpr (PC) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tmem + TM::S0 + (g & 1) * NR, tmem + TM::K0 + (g & 1) * 64 + 8 * kk,
                     sdesc_k128(qb + SM::kQlo - SM::kQ + (kk >> 2) * NR * 128 + (kk & 3) * 32), idesc, 1u);
          }
          tc_commit(&sfull[g & 1]);
        }
        ++commits[g & 1];
        if (lane == 0) trace_ev(p, g, 8);
      } else {
        if (!mwait(&pready[g & 3], (g >> 2) & 1) || !mwait(&vready[g & 1], (g >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t pb = p_s + (g & 3) * kPBufBytes;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)   // positions 16kk .. 16kk+15: two 8-position swizzle atoms of 1 KB
            mma_ts(tmem + TM::O0 + ((c.it - item_begin) & 1) * NR, tmem + TM::V0 + (g & 1) * 64 + 8 * kk,
                   sdesc_mn128(pb + kk * 2048, kPBufBytes, 1024), idesc, (c.i > 0 || kk > 0) ? 1u : 0u);
          tc_commit(&pvdone[g & 3]);
        }
        ++commits[g & 3];
        if (lane == 0) trace_ev(p, g, 9);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) {
      if (!*abort_any) record_status(p.status, PA_ERR_DEVICE_TIMEOUT, item_begin);
      *abort_any = 1;
    }
    // drain: every MMA this warp issued completes before TMEM is released
    for (int j = 0; j < kPBufs; ++j)
      if (commits[j]) mbar_wait(is_s ? &sfull[j] : &pvdone[j], (commits[j] - 1) & 1, kDrainNs);
  } else if (wg == 4) {
    // the last warp has no role (it completes the warpgroup)
  } else if (wg == 1 && p.softmax_wgs == 1) {
    // every item's rows are in the first half: this warpgroup has no rows
  } else if (wg < 2) {
    // ================================================================ softmax
    // warpgroup wg owns packed rows [r_lo, r_lo + NH); lane = position
    const int r_lo = wg * NH;
    const int bar_id = 1 + wg;
    const int pos_in_tile = tid & 127;
    volatile int* my_abort = abort_grp + wg;
    bool fail = false, stop = false;
    auto note_fail = [&](int it) {
      if (!*abort_any) record_status(p.status, PA_ERR_DEVICE_TIMEOUT, it);
      *abort_any = 1;
      *my_abort = 1;
      fail = true;
    };
    // epilogue of local item li (last tile gl) for this warpgroup's rows:
    // O^T row d = this thread's TMEM lane, times 1/l and the V scale
    auto epilogue = [&](int li, uint32_t gl) -> bool {
      const int it = item_begin + li;
      const Item m = isrc.at(it);
      // a failed wait is published through the warpgroup's abort flag and
      // acted on after the named barrier below, so that every thread of the
      // warpgroup reaches that barrier
      if (!fail && !dwait(&pvdone[gl & 3], (gl >> 2) & 1, limit, abort_any)) note_fail(it);
      tc_fence_after();
      // O^T columns (thread = head dim d) are staged as fp32 [j][d], 16 rows
      // per pass, in the P^T slot of tile gl: PV_gl has completed, and that
      // slot is written again only for tile gl + 4, whose S needs both
      // warpgroups to have read S of tile gl + 2, i.e. to be past this
      // epilogue.  Warpgroup wg uses bytes [8 KB wg, 8 KB wg + 8 KB).  The rows
      // then leave as 16-byte pieces from a rolled loop that applies 1/l, the
      // V scale and the output epilogue: this code runs at about the same
      // moment in every CTA and is kept small.
      const int d = pos_in_tile;
      const int n_rows = m.ntok * G;
      float* stg = reinterpret_cast<float*>(smem + SM::kP + (gl & 3) * kPBufBytes + wg * 8192);
      const float* inv = lsum_s + (li & 1) * NR;
      const bool per_channel = p.scale_kind == PA_SCALE_PER_CHANNEL;
      const float vs_head = per_channel ? 1.0f : vscale(m.kvh);
      const bool vec = m.nch > 1 || (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
      uint32_t v[NH];
#pragma unroll
      for (int c = 0; c < NH / 8; ++c)
        tmem_ld8(t_lane + TM::O0 + (li & 1) * NR + r_lo + 8 * c,
                 *reinterpret_cast<uint32_t(*)[8]>(&v[8 * c]));
      tmem_wait_ld();
      tc_fence_before();
      // rows j0 .. j0 + nj - 1 of this warpgroup, from the staging buffer
      auto write_rows = [&](int j0, int nj) {
#pragma unroll 1
        for (int q = pos_in_tile; q < nj * 16; q += 128) {
          const int j = q >> 4, c = q & 15;   // row r_lo + j0 + j, dims 8c .. 8c+7
          const int r = r_lo + j0 + j;
          if (r >= n_rows) continue;
          const float4 a = *reinterpret_cast<const float4*>(stg + j * kHeadDim + 8 * c);
          const float4 b = *reinterpret_cast<const float4*>(stg + j * kHeadDim + 8 * c + 4);
          float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          const float sc = inv[r] * vs_head;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            f[k] *= per_channel ? sc * load_scale(p.v_scale, p.scale_kind, m.kvh * kHeadDim + 8 * c + k) : sc;
          const int token = m.tok0 + r / G;
          const int head = m.kvh * G + r % G;
          if (m.nch == 1) {
            const int64_t o = ((int64_t)token * p.q_heads + head) * kHeadDim + 8 * c;
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = ep_value(p.ep, f[k], head * kHeadDim + 8 * c + k);
            if (p.ep.int8_out) {
              int8_t* dst = reinterpret_cast<int8_t*>(p.out) + o;
              if (vec) {
                uint32_t w0 = 0, w1 = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  w0 |= ep_int8(p.ep, f[k]) << (8 * k);
                  w1 |= ep_int8(p.ep, f[4 + k]) << (8 * k);
                }
                *reinterpret_cast<uint2*>(dst) = make_uint2(w0, w1);
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) dst[k] = (int8_t)ep_int8(p.ep, f[k]);
              }
            } else if (vec) {
              *reinterpret_cast<uint4*>(p.out + o) =
                  make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                             pack_bf16x2(f[6], f[7]));
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) p.out[o + k] = __float2bfloat16_rn(f[k]);
            }
          } else {
            const int64_t sp = (int64_t)(m.chunk + (token - m.tok0) * m.nch) * p.q_heads + head;
            float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.part_o) + sp * kHeadDim + 8 * c);
            dst[0] = make_float4(f[0], f[1], f[2], f[3]);
            dst[1] = make_float4(f[4], f[5], f[6], f[7]);
          }
        }
      };
      constexpr int kP0 = NH < 16 ? NH : 16;   // rows of the first pass
#pragma unroll
      for (int j = 0; j < kP0; ++j) stg[j * kHeadDim + d] = __uint_as_float(v[j]);
      bar_sync(bar_id, 128);
      if (*my_abort) return false;
      write_rows(0, kP0);
      if constexpr (NH > kP0) {
        bar_sync(bar_id, 128);   // the first pass has read the staging buffer
#pragma unroll
        for (int j = kP0; j < NH; ++j) stg[(j - kP0) * kHeadDim + d] = __uint_as_float(v[j]);
        bar_sync(bar_id, 128);
        write_rows(kP0, NH - kP0);
      }
      if (tid == 0) trace_ev(p, gl, 10);
      return true;
    };
    int pend_li = -1;
    uint32_t pend_g = 0;
    uint32_t g = 0;
    float l[NH];
    for (int it = item_begin; it < item_end && !stop; ++it) {
      const Item cur = isrc.at(it);
      const int li = it - item_begin;
      const int n_rows = cur.ntok * G;
      const float c_log2 = p.sm_scale_log2 * kFold8<FP4> *
          (p.scale_kind == PA_SCALE_PER_CHANNEL ? 1.0f : kscale(cur.kvh));
      const uint32_t o_col = TM::O0 + (li & 1) * NR + r_lo;
      // speculative tree mask: the item's first token within its sequence and
      // the sequence's cached prefix length (appended positions start there)
      int tok0_local = 0, pre_len = 0;
      const uint8_t* tmask = nullptr;
      if constexpr (TREE) {
        tok0_local = cur.tok0 - p.cu_seqlens_q[cur.b];
        pre_len = cur.cbase - tok0_local;
        tmask = p.attn_mask + (int64_t)cur.b * p.mask_dim * p.mask_dim;
      }
#pragma unroll
      for (int j = 0; j < NH; ++j) l[j] = 0.0f;
      bool m_ninf = false;   // some row of this half has m = -inf (warpgroup-uniform)
      for (int i = 0; i < cur.ntiles; ++i, ++g) {
        // ---- S_g columns of this half -> registers, then release the S buffer
        float s[NH];
        if (!fail && !dwait(&sfull[g & 1], (g >> 1) & 1, limit, abort_any)) note_fail(it);
        tc_fence_after();
        if (tid == 0) trace_ev(p, g, 3);
        if (!fail) {
          uint32_t v[NH];
#pragma unroll
          for (int c = 0; c < NH / 8; ++c)
            tmem_ld8(t_lane + TM::S0 + (g & 1) * NR + r_lo + 8 * c,
                     *reinterpret_cast<uint32_t(*)[8]>(&v[8 * c]));
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < NH; ++j) s[j] = __uint_as_float(v[j]);
        } else {
#pragma unroll
          for (int j = 0; j < NH; ++j) s[j] = 0.f;
        }
        tc_fence_before();
        warp_arrive(&sfree[g & 1], lane);

        // ---- x = s * c - m: log2 units, relative to the row's running max m,
        // -inf where masked.  The first tile of an item, and every tile while
        // some row of this half has seen no visible position yet (m = -inf),
        // take the general path, which forms x once the new maximum is known.
        const int tpos0 = cur.kv0 + i * kTileTok;
        const int jpos = tpos0 + pos_in_tile;
        const bool need_mask = (tpos0 + kTileTok > cur.kv1) || (tpos0 + kTileTok - 1 > cur.cbase) ||
                               (TREE && tpos0 + kTileTok > pre_len);
        const bool general = (i == 0) || m_ninf;
        const float4* m4s = reinterpret_cast<const float4*>(m_s + r_lo);
        bool exceed = general;
        if (need_mask) {
          const int lim_tok = jpos - cur.cbase;   // visible for rows of token >= lim_tok
          const bool tree = TREE && jpos >= pre_len && jpos < cur.kv1;
#pragma unroll
          for (int j = 0; j < NH; ++j) {
            bool vis = (jpos < cur.kv1) && (r_lo + j >= lim_tok * G);
            if (tree && vis && r_lo + j < n_rows) {
              // draft token (row's token) sees appended token jpos - pre_len?
              const int tl = tok0_local + (r_lo + j) / G;
              vis = tmask[tl * p.mask_dim + (jpos - pre_len)] != 0;
            }
            s[j] = vis ? s[j] * c_log2 : -INFINITY;
          }
          if (!general) {
#pragma unroll
            for (int j4 = 0; j4 < NH / 4; ++j4) {
              const float4 m4 = m4s[j4];
              const float mv[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                s[4 * j4 + e] -= mv[e];
                exceed |= s[4 * j4 + e] > kTau;
              }
            }
          }
        } else if (!general) {
#pragma unroll
          for (int j4 = 0; j4 < NH / 4; ++j4) {
            const float4 m4 = m4s[j4];
            const float mv[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[4 * j4 + e] = fmaf(s[4 * j4 + e], c_log2, -mv[e]);
              exceed |= s[4 * j4 + e] > kTau;
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < NH; ++j) s[j] *= c_log2;
        }
        // padded rows have Q' = 0, so x = 0 - 0 there and they never exceed
        const bool resc = bar_or(bar_id, 128, exceed);
        if (*my_abort) { fail = true; stop = true; break; }
        if (resc) {
          if (!general) {
            // back to s * c (-inf stays -inf)
#pragma unroll
            for (int j4 = 0; j4 < NH / 4; ++j4) {
              const float4 m4 = m4s[j4];
              s[4 * j4 + 0] += m4.x;
              s[4 * j4 + 1] += m4.y;
              s[4 * j4 + 2] += m4.z;
              s[4 * j4 + 3] += m4.w;
            }
          }
          // exact tile maximum per row, new running max; rescale l (registers)
          // and this half's columns of O (TMEM) by 2^(m_old - m_new).  Up to
          // 24 rows per warpgroup the warp maxima come from the halving
          // exchange (48 rows: 5 % faster than one redux.sync per row)
          if constexpr (NH <= 24) {
            constexpr int kLeft = sum_rows_left<NH>();
            constexpr int kDup = 32 * kLeft / NH;
            float t[NH / 2];
            int row0 = 0;
            max_rows_first<NH>(s, t, lane, row0);
            if ((lane & (kDup - 1)) == 0) {
#pragma unroll
              for (int k = 0; k < kLeft; ++k) red[(warp & 3) * NR + r_lo + row0 + k] = t[k];
            }
          } else {
#pragma unroll
            for (int j = 0; j < NH; ++j) {
              const float wm = warp_max(s[j]);
              if (lane == 0) red[(warp & 3) * NR + r_lo + j] = wm;
            }
          }
          bar_sync(bar_id, 128);
          if (pos_in_tile < NH) {
            const int r = r_lo + pos_in_tile;
            float a = 1.0f, mn = 0.0f;   // padded rows keep m = 0
            if (r < n_rows) {
              const float mo = (i == 0) ? -INFINITY : m_s[r];
              const float tm = fmaxf(fmaxf(red[r], red[NR + r]), fmaxf(red[2 * NR + r], red[3 * NR + r]));
              mn = fmaxf(mo, tm);
              a = (mo == -INFINITY) ? 0.0f : fast_exp2(mo - mn);
            }
            m_s[r] = mn;
            alpha_s[r] = a;
          }
          bar_sync(bar_id, 128);
          if (i > 0) {
#pragma unroll
            for (int j = 0; j < NH; ++j) l[j] *= alpha_s[r_lo + j];
            // O holds PV of the earlier tiles of this item: wait for the last one
            if (!fail && !dwait(&pvdone[(g - 1) & 3], ((g - 1) >> 2) & 1, limit, abort_any))
              note_fail(it);
            tc_fence_after();
            if (!fail) {
#pragma unroll
              for (int c = 0; c < NH / 8; ++c) {
                uint32_t v[8];
                tmem_ld8(t_lane + o_col + 8 * c, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha_s[r_lo + 8 * c + j]);
                tmem_st8(t_lane + o_col + 8 * c, v);
              }
              tmem_wait_st();
            }
          }
          // x against the new maximum; a row with no visible position so far
          // (m = -inf) has only x = -inf
          m_ninf = false;
#pragma unroll
          for (int j4 = 0; j4 < NH / 4; ++j4) {
            const float4 m4 = m4s[j4];
            const float mv[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              m_ninf |= mv[e] == -INFINITY;
              s[4 * j4 + e] -= mv[e] == -INFINITY ? 0.0f : mv[e];
            }
          }
          bar_sync(bar_id, 128);  // red / alpha_s / m_s are reused by the next rescale
        }
        // P^T slot g&3 was last read by PV_{g-4}
        if (g >= kPBufs && !fail &&
            !dwait(&pvdone[g & 3], ((g - kPBufs) >> 2) & 1, limit, abort_any))
          note_fail(it);
        if (tid == 0) trace_ev(p, g, 11);
        {
          // p = 2^x (0 where masked); this position's row of P^T: 16-byte
          // chunk c (rows 8c .. 8c+7) at chunk c ^ (position & 7)
          const int prw = KV == PA_KV_INT4 ? 2 * (pos_in_tile & 3) + ((pos_in_tile >> 2) & 1) : pos_in_tile & 7;
          const uint32_t prow = p_s + (g & 3) * kPBufBytes + (pos_in_tile >> 3) * 1024 + prw * 128;
#pragma unroll
          for (int cc = 0; cc < NH / 8; ++cc) {
            float pv[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              pv[e] = fast_exp2(s[8 * cc + e]);
              l[8 * cc + e] += pv[e];
            }
            const int chunk = wg * (NH / 8) + cc;
            st_shared_v4(prow + ((chunk ^ prw) << 4),
                         make_uint4(pack_half2(pv[0], pv[1]), pack_half2(pv[2], pv[3]),
                                    pack_half2(pv[4], pv[5]), pack_half2(pv[6], pv[7])));
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        warp_arrive(&pready[g & 3], lane);
        if (tid == 0) trace_ev(p, g, 4);
        // epilogue of the previous item, one tile after its last PV was queued
        if (pend_li >= 0 && pend_li < li) {
          if (!epilogue(pend_li, pend_g)) { stop = true; break; }
          pend_li = -1;
        }
        if (i + 1 == cur.ntiles) {
          // row sums over all positions of the item: warp, then warpgroup; the
          // owner thread of row r keeps 1/l and writes the row statistics.
          // Up to 24 rows per warpgroup the halving exchange is used (48 rows:
          // 27 shuffles a thread instead of 120); at 32 rows it measured
          // slower than one butterfly per row (more spilled registers)
          if constexpr (NH <= 24) {
            constexpr int kLeft = sum_rows_left<NH>();
            constexpr int kDup = 32 * kLeft / NH;   // lanes holding the same rows
            int row0 = 0;
            sum_rows_step<NH, 16>(l, lane, row0);
            if ((lane & (kDup - 1)) == 0) {
#pragma unroll
              for (int k = 0; k < kLeft; ++k) red_l[(warp & 3) * NR + r_lo + row0 + k] = l[k];
            }
          } else {
#pragma unroll
            for (int j = 0; j < NH; ++j) {
              float v = l[j];
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
              if (lane == 0) red_l[(warp & 3) * NR + r_lo + j] = v;
            }
          }
          bar_sync(bar_id, 128);
          if (pos_in_tile < NH) {
            const int r = r_lo + pos_in_tile;
            const float lr = red_l[r] + red_l[NR + r] + red_l[2 * NR + r] + red_l[3 * NR + r];
            lsum_s[(li & 1) * NR + r] = lr > 0.f ? __frcp_rn(lr) : 0.f;
            if (r < n_rows) {
              const int token = cur.tok0 + r / G;
              const int head = cur.kvh * G + r % G;
              const float mr = m_s[r];
              const float ln2 = 0.69314718055994530942f;
              if (cur.nch == 1) {
                if (p.lse != nullptr)
                  p.lse[(int64_t)token * p.q_heads + head] =
                      lr > 0.f ? (mr + __log2f(lr)) * ln2 : -INFINITY;
              } else {
                const int64_t sp = (int64_t)(cur.chunk + (token - cur.tok0) * cur.nch) * p.q_heads + head;
                p.part_m[sp] = lr > 0.f ? mr * ln2 : -INFINITY;
                p.part_d[sp] = lr;
              }
            }
          }
          bar_sync(bar_id, 128);  // 1/l of this item visible to the warpgroup
          pend_li = li;
          pend_g = g;
        }
      }
    }
    if (!stop && pend_li >= 0) epilogue(pend_li, pend_g);
  } else {
    // ================================================================ CV warpgroup
    // Q' of each item, K rows (lane = position) and V^T rows (lane = head dim)
    // into TMEM
    // This warpgroup runs ahead of the softmax, so its waits suspend for the
    // hardware's default time rather than re-probing every 32 ns (fewer issue
    // slots taken from the softmax warps on the same sub-partitions).
    const int d = tid & 127;  // TMEM lane: K position / V head dim / output dim
    const bool do_k = wg == 2, do_v = wg == 3;
    uint32_t g = 0;
    bool fail = false;
    auto note_fail = [&](int it) {
      if (!*abort_any) record_status(p.status, PA_ERR_DEVICE_TIMEOUT, it);
      *abort_any = 1;
      fail = true;
    };
    // Q' of an item -> shared memory buffer qb (fp16, K-major, 128B swizzle, padded rows zero)
    // A thread's pieces are rows d/16 + 8k, dims 8 (d & 15) .. +7: every
    // load is issued before the first conversion, so their latencies overlap
    // (a shared-memory store between two loads would order them).
    auto load_q = [&](const Item& m, uint32_t qb) {
      constexpr int kPieces = NR * 16 / 128;
      static_assert(NR * 16 % 128 == 0, "whole 16-byte pieces per thread");
      const int n_rows = m.ntok * G;
      const int ch = d & 15;
      uint4 raw[kPieces];
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int r = (d >> 4) + 8 * k;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (r < n_rows) {
          const int token = m.tok0 + r / G;
          const int head = m.kvh * G + r % G;
          raw[k] = *reinterpret_cast<const uint4*>(p.q + (int64_t)token * p.q_stride +
                                                   head * kHeadDim + ch * 8);
        }
      }
      // per-channel K scales of these 8 dims (1 otherwise: x * 1 is exact)
      float sc[8];
      if (p.scale_kind == PA_SCALE_PER_CHANNEL) {
        const uint4 sr = *reinterpret_cast<const uint4*>(
            reinterpret_cast<const __nv_bfloat16*>(p.k_scale) + m.kvh * kHeadDim + ch * 8);
        const __nv_bfloat16* sv = reinterpret_cast<const __nv_bfloat16*>(&sr);
#pragma unroll
        for (int e = 0; e < 8; ++e) sc[e] = __bfloat162float(sv[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) sc[e] = 1.0f;
      }
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int r = (d >> 4) + 8 * k;
        uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};   // lo: PC only
        if (r < n_rows) {
          const __nv_bfloat16* hv = reinterpret_cast<const __nv_bfloat16*>(&raw[k]);
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __bfloat162float(hv[e]) * sc[e];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = f[pair_first<KV>(e)], b = f[pair_first<KV>(e) + pair_gap<KV>()];
            hi[e] = pack_half2(a, b);
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi[e]));
            if constexpr (PC) lo[e] = pack_half2(a - h.x, b - h.y);
          }
        }
        const uint32_t dst = qb + (ch >> 3) * NR * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
        st_shared_v4(dst, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        if constexpr (PC)
          st_shared_v4(dst + SM::kQlo - SM::kQ, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
      fence_proxy_async_smem();
    };
    int q_ahead = -1;   // item whose Q' was written during the previous item
    for (int it = item_begin; it < item_end && !fail; ++it) {
      const Item m = isrc.at(it);
      const int li = it - item_begin;
      for (int i = 0; i < m.ntiles; ++i, ++g) {
        const int stage = g % kStages;
        // K buffer g&1 was last read by S_{g-2}; Q' buffer li&1 by the S of item
        // li-2, whose last tile is at most g-2
        if (do_k && g >= 2 && !wait_or_abort(&sfull[g & 1], ((g - 2) >> 1) & 1, limit, abort_any)) {
          note_fail(it);
          break;
        }
        if (do_k) tc_fence_after();   // the K stores below come after the MMAs that read the buffer
        if (do_k && i == 0) {
          if (q_ahead != it) load_q(m, q_s + (li & 1) * NR * 256);
          // the next item's query rows into L2 now; its Q' is written at this
          // item's second tile (below), so that no item boundary waits for it
          if (it + 1 < item_end) {
            const Item mn = isrc.at(it + 1);
            const int rows = mn.ntok * G;
            if (d < 2 * rows) {
              const int r = d >> 1;
              prefetch_l2(p.q + (int64_t)(mn.tok0 + r / G) * p.q_stride + (mn.kvh * G + r % G) * kHeadDim +
                          64 * (d & 1));
            }
          }
        }
        if (do_k && i == 1 && it + 1 < item_end) {
          // Q' buffer (li + 1) & 1 was last read by the S of item li - 1, whose
          // last tile is g - 2 or earlier
          load_q(isrc.at(it + 1), q_s + ((li + 1) & 1) * NR * 256);
          q_ahead = it + 1;
        }
        if (!wait_or_abort(&full[stage], (g / kStages) & 1, limit, abort_any)) { note_fail(it); break; }
        if (do_k && d == 0) trace_ev(p, g, 1);
        if (!do_k) {
          // this warpgroup converts V only
        } else {
          // position d: code row 36 (half page) + row of its page's box, its eight
          // block scales in one of the rows behind the half's codes
          const uint32_t kbase = s_base + stage * kStageBytes + (d >> 6) * kSlot4;
          const int hrow = ((d >> 5) & 1) * (kV4HalfBytes / 64), r = hrow + (d & 31);
          const int rs = hrow + kV4Half + ((d & 31) >> 3);
          const uint2 sw = ld_shared_v2(kbase + rs * 64 + ((((d & 7) >> 1) ^ ((rs >> 1) & 3)) << 4) + 8 * (d & 1));
          uint4 nx = ld_shared_v4(kbase + r * 64 + (((r >> 1) & 3) << 4));
          const uint32_t dst = t_lane + TM::K0 + (g & 1) * 64;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {   // dims 32c .. 32c+31
            uint32_t s[2], n[2][2], x[16];
            scale_pair_fold8<FP4>((uint16_t)((c < 2 ? sw.x : sw.y) >> (16 * (c & 1))), s, n);
            const uint4 rc = nx;
            nx = ld_shared_v4(kbase + r * 64 + ((((c + 1) & 3) ^ ((r >> 1) & 3)) << 4));
            const uint32_t w[4] = {rc.x, rc.y, rc.z, rc.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t y[4];
              codes8<FP4>(w[k], y);
#pragma unroll
              for (int i = 0; i < 4; ++i) x[4 * k + i] = scaled_fold8<FP4>(y[i], s[k >> 1], n[k >> 1][i & 1]);
            }
            tmem_st16(dst + 16 * c, x);
          }
          tmem_wait_st();
        }
        if (do_k) {
          warp_arrive(&empty[stage], lane);
          tc_fence_before();
          warp_arrive(&kready[g & 1], lane);
          if (d == 0) trace_ev(p, g, 2);
        }
        if (!do_v) continue;
        // V buffer g&1 was last read by PV_{g-2}
        if (g >= 2 && !wait_or_abort(&pvdone[(g - 2) & 3], ((g - 2) >> 2) & 1, limit, abort_any)) {
          note_fail(it);
          break;
        }
        tc_fence_after();
        if (d == 0) trace_ev(p, g, 5);
        {
          // V^T row d of tile g.  The warp's two scale blocks (32 dims) are turned
          // into fp16 once: lane (b, k) takes positions 8k .. 8k+7 of block b; 0
          // past kv1, where the bytes may hold anything.
          const int nvalid = min(kTileTok, m.kv1 - (m.kv0 + i * kTileTok));
          const uint32_t vst = s_base + stage * kStageBytes + kVOff;
          const uint32_t scr = s_base + SM::kVs16 + (warp & 3) * kVs16Warp;
          {
            const int blk = lane >> 4, k = lane & 15;   // k: 8-position group of the tile
            uint2 sw = ld_shared_v2(vst + (k >> 3) * kSlot4 + ((k >> 2) & 1) * kV4HalfBytes + kV4Codes +
                                    (2 * (warp & 3) + blk) * kV4Half + 8 * (k & 3));
            keep_scales(sw, nvalid - 8 * k);
            uint32_t f[4];
            scales8<FP4>(sw, f);
            st_shared_v4(scr + (blk * 16 + k) * 16, make_uint4(f[0], f[1], f[2], f[3]));
            __syncwarp();
          }
          const uint32_t dst = t_lane + TM::V0 + (g & 1) * 64;
#pragma unroll
          for (int c = 0; c < 4; ++c) {   // half page: positions 32c .. 32c+31
            const uint4 r4 = ld_shared_v4(vst + (c >> 1) * kSlot4 + (c & 1) * kV4HalfBytes + d * (kV4Half / 2));
            const uint32_t w[4] = {r4.x, r4.y, r4.z, r4.w};
            uint32_t x[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 sv = ld_shared_v4(scr + ((lane >> 4) * 16 + 4 * c + k) * 16);
              const uint32_t sc[4] = {sv.x, sv.y, sv.z, sv.w};
              uint32_t y[4];
              codes8<FP4>(w[k], y);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[4 * k + e] = scaled<FP4>(y[e], sc[e], e);
            }
            tmem_st16(dst + 16 * c, x);
          }
          tmem_wait_st();
          __syncwarp();   // every lane has read the scales before the next tile writes them
        }
        warp_arrive(&empty[stage], lane);
        if (d == 0) trace_ev(p, g, 6);
        tc_fence_before();
        warp_arrive(&vready[g & 1], lane);
        if (d == 0) trace_ev(p, g, 7);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();   // the merge grid may be scheduled while the last CTAs finish
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace pa
