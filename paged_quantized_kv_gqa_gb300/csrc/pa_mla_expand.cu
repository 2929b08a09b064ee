// pa_mla_expand.cu - keys and values of every head from many latent rows, CTA pairs
// (tcgen05 cta_group::2), sm_103a:  [k | v][n][h] = [W_k; W_v][h] c[n], 512 -> 128 + 128.
//
// A pair makes 256 rows x 256 outputs of one head.  Its CTAs hold a half of the head's
// weights each (CTA 0 W_k, CTA 1 W_v, all 512 dims: 128 KB) and stream 128 rows of c each,
// 64 dims a stage.  A pair's MMA reads both CTAs' halves, so that an SM takes in 32 bytes a
// cycle at the tensor cores' rate; a CTA by itself with a 128 x 256 tile takes 96.  Two
// accumulators of 256 columns: a tile's rows leave (bf16, by way of shared memory and TMA)
// while the next one is made.
// The tiles, row blocks fastest, are cut into equal runs, one a pair.  (With the rows
// resident and heads fastest the scattered writes of 8192 rows of 128 heads, 537 MB, took
// 185 us without any MMA, in this order 171; the whole kernel 212 and 191.)
// Bound: the tensor cores (512 flops a byte) by their nominal rates; in fact the writes, whose
// rate is about 3.9 TB/s when nothing else is done (a fill of 537 MB).
#include "pa_common.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;                   // rows of a CTA
constexpr int kBlk = 16384;                  // 128 rows x 64 dims
constexpr int kKBlocks = 8;
constexpr int kStages = 4;
constexpr int kThreads = 320;                // epilogue warps 0-7, TMA warp 8, MMA warp 9

struct Smem {
  static constexpr int kB = 0;                              // [8][128 outputs][128 B]
  static constexpr int kA = kB + kKBlocks * kBlk;           // [stage][128 rows][128 B]
  static constexpr int kOut = kA + kStages * kBlk;          // [K, V][128 rows][128 B]
  static constexpr int kBars = kOut + 2 * kBlk;             // full[S] empty[S] bfull bfree dfull[2] dfree[2] drain
  static constexpr int kMisc = kBars + (2 * kStages + 7) * 8;
  static constexpr int kTotal = kMisc + 16 + 1024;
  static_assert(kTotal <= 232448, "shared memory overflow");
};

struct ExpandParams {
  int32_t* status;
  int64_t wait_limit_ns;
  int32_t blocks, pairs;   // blocks of 256 rows, CTA pairs
  int64_t tiles;
  int32_t skip_first_load;
};

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_expand_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const ExpandParams p) {
  using SM = Smem;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBars);   // of CTA 0: both CTAs' bytes
  uint64_t* empty = full + kStages;    // of each CTA
  uint64_t* bfull = empty + kStages;   // of CTA 0
  uint64_t* bfree = bfull + 1;         // of each CTA
  uint64_t* dfull = bfree + 1;         // [accumulator], of each CTA
  uint64_t* dfree = dfull + 2;         // [accumulator], of CTA 0: both CTAs' epilogue warps
  uint64_t* drain = dfree + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kMisc);
  volatile int* abort_any = reinterpret_cast<volatile int*>(smem + SM::kMisc + 4);
  const uint32_t s_base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int64_t pair = blockIdx.x >> 1;
  const int64_t begin = p.tiles * pair / p.pairs, end = p.tiles * (pair + 1) / p.pairs;
  const uint64_t limit = (uint64_t)p.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(bfull, 1);
    mbar_init(bfree, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&dfull[b], 1);
      mbar_init(&dfree[b], 16);
    }
    mbar_init(drain, 1);
    *abort_any = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();   // both CTAs' barriers are there before any remote access
  const uint32_t tmem = *tmem_slot;
  const uint32_t peer_abort = mapa_shared(smem_u32((const void*)abort_any), rank ^ 1u);
  auto raise = [&](int64_t t) {
    if (!*abort_any) record_status(p.status, PA_ERR_DEVICE_TIMEOUT, (int)t);
    *abort_any = 1;
    st_cluster_u32(peer_abort, 1u);
  };

  if (warp == 8) {
    // ================================================================ TMA (both CTAs)
    if (lane == 0) {
      tma_prefetch_desc(&tm_x);
      tma_prefetch_desc(&tm_w);
      const uint32_t full0 = mapa_shared(smem_u32(full), 0), bfull0 = mapa_shared(smem_u32(bfull), 0);
      uint32_t n = 0, nb = 0;   // blocks of rows, loads of weights
      int64_t loaded = -1;
      bool ok = true;
      for (int64_t t = begin; t < end && ok; ++t) {
        const int64_t head = t / p.blocks;
        const int row = (int)(t - head * p.blocks) * 2 * kRows + (int)rank * kRows;
        if (head != loaded) {
          if (nb > 0 && !wait_or_abort(bfree, (nb - 1) & 1, limit, abort_any)) {
            raise(t);
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(bfull, 2 * kKBlocks * kBlk);
          for (int kb = 0; kb < kKBlocks; ++kb)
            tma_load_3d_pair(smem + SM::kB + kb * kBlk, &tm_w, bfull0, 64 * kb, (int)rank * 128, (int)head);
          loaded = head;
          ++nb;
        }
        for (int kb = 0; kb < kKBlocks; ++kb, ++n) {
          const uint32_t s = n % kStages;
          if (n >= kStages && !wait_or_abort(&empty[s], (n / kStages - 1) & 1, limit, abort_any)) {
            raise(t);
            ok = false;
            break;
          }
          if (p.skip_first_load && n == 0 && rank == 0) continue;   // failure-detection test hook
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kBlk);
          tma_load_3d_pair(smem + SM::kA + s * kBlk, &tm_x, full0 + 8 * s, 64 * kb, 0, row);
        }
      }
      if (ok) {
        // every load has landed once the MMAs that read it are done
        for (uint32_t k = n > kStages ? n - kStages : 0; k < n; ++k)
          if (!wait_or_abort(&empty[k % kStages], (k / kStages) & 1, limit, abort_any)) ok = false;
        if (!ok) raise(end);
      }
    }
  } else if (warp == 9) {
    // ================================================================ MMA (CTA 0, for both)
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(256, 256) | (1u << 7) | (1u << 10);
      const uint64_t b = sdesc_k128(s_base + SM::kB);
      uint32_t n = 0, nb = 0, d = 0;
      int64_t loaded = -1;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = wait_or_abort(bar, parity, limit, abort_any, whole_warp);
        tc_fence_after();
        return ok;
      };
      int64_t t = begin;
      for (; t < end; ++t, ++d) {
        const int64_t head = t / p.blocks;
        if (head != loaded) {
          if (!wait(bfull, nb & 1)) break;
          ++nb;
          loaded = head;
        }
        if (d >= 2 && !wait(&dfree[d & 1], ((d >> 1) - 1) & 1)) break;
        const uint32_t acc = tmem + 256 * (d & 1);
        const bool head_follows = t + 1 < end && (t + 1) / p.blocks != head;
        for (int kb = 0; kb < kKBlocks; ++kb, ++n) {
          const uint32_t s = n % kStages;
          if (!wait(&full[s], (n / kStages) & 1)) break;
          const uint64_t a = sdesc_k128(s_base + SM::kA + s * kBlk);
          if (elect_one()) {
#pragma unroll
            for (int kq = 0; kq < 4; ++kq)
              mma_ss_pair(acc, a + ((32 * kq) >> 4), b + ((kb * kBlk + 32 * kq) >> 4), idesc, (kb | kq) ? 1u : 0u);
            tc_commit_pair(&empty[s]);
            if (kb + 1 == kKBlocks) {
              tc_commit_pair(&dfull[d & 1]);
              if (head_follows) tc_commit_pair(bfree);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) raise(t);
      // every MMA issued completes before TMEM is released (in both CTAs: CTA 1 comes to that
      // behind the cluster barrier)
      if (elect_one()) tc_commit_pair(drain);
      __syncwarp();
      mbar_wait(drain, 0, kDrainNs);
    }
  } else {
    // ================================================================ epilogue (both CTAs)
    // warps 0-3 the keys' 128 columns, 4-7 the values', 32 rows each (4 warps for all 256
    // columns were slower than the MMAs)
    const int row = 32 * (warp & 3), side = warp >> 2;
    const uint32_t t_lane = tmem + ((uint32_t)row << 16) + 128 * side;
    const uint32_t dfree0 = mapa_shared(smem_u32(dfree), 0);
    const uint32_t box = s_base + SM::kOut + side * kBlk + row * 128, line = box + lane * 128;
    const CUtensorMap* map = side ? &tm_v : &tm_k;
    uint32_t d = 0;
    for (int64_t t = begin; t < end; ++t, ++d) {
      const int head = (int)(t / p.blocks);
      const int r0 = (int)(t - (int64_t)head * p.blocks) * 2 * kRows + (int)rank * kRows + row;
      if (!wait_or_abort(&dfull[d & 1], (d >> 1) & 1, limit, abort_any, whole_warp)) {
        if (lane == 0) raise(t);
        break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int j = 0; j < 2; ++j) {
        uint32_t v[64];
        tmem_ld32(t_lane + 256 * (d & 1) + 64 * j, v);
        tmem_ld32(t_lane + 256 * (d & 1) + 64 * j + 32, v + 32);
        tmem_wait_ld();
        if (j == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(dfree0 + 8 * (d & 1));
        }
        if (lane == 0) bulk_store_drain();   // the last store has read the buffer
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(v[8 * c + 2 * k]), __uint_as_float(v[8 * c + 2 * k + 1]));
            w[k] = *reinterpret_cast<uint32_t*>(&h2);
          }
          st_shared_v4(line + ((c ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tma_store_3d(map, box, 64 * j, head, r0);
      }
    }
    if (lane == 0) bulk_store_drain();   // shared memory is read before the CTA leaves
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();   // no CTA leaves while its peer may still signal or read it
  // nor before the MMAs' own signals have come, which the barrier above does not order.  drain's
  // is the last of them; roles that gave up did not wait for theirs, nor for loads counted in the
  // other CTA: a time that they all take.
  if (warp == 9) {
    mbar_wait(drain, 0, kDrainNs);
    if (*abort_any) {
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 1000000ull) {
      }
    }
  }
  if (warp == 0) tmem_dealloc_pair(tmem, 512);
}

cudaError_t launch_mla_expand(const MlaProduct& m, const FaultCfg& fc, int num_sms, cudaStream_t stream) {
  ExpandParams p{};
  p.status = m.status;
  p.wait_limit_ns = fc.wait_limit_ns;
  p.skip_first_load = fc.skip_first_load;
  p.blocks = (int32_t)(((int64_t)m.rows + 2 * kRows - 1) / (2 * kRows));
  p.tiles = (int64_t)p.blocks * m.heads;
  p.pairs = (int32_t)(p.tiles < num_sms / 2 ? p.tiles : num_sms / 2);
  const cudaError_t e = cudaFuncSetAttribute(mla_expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::kTotal);
  if (e != cudaSuccess) return e;
  mla_expand_kernel<<<2 * p.pairs, kThreads, Smem::kTotal, stream>>>(m.tm[0], m.tm[1], m.tm[2], m.tm[3], p);
  return cudaGetLastError();
}

}  // namespace pa
