// pa_mla_product.cu - the products around latent attention, tcgen05 + TMA, sm_103a:
//   absorb   q'[t][h] = q_nope[t][h] W_k[h]   (128 -> 512; the rotated 64 dims copied)
//   project  o[t][h] = W_v[h] o'[t][h]        (512 -> 128)
//   expand   k[n][h] = W_k[h] c[n], v[n][h] = W_v[h] c[n]   (512 -> 128 + 128)
//
// A CTA makes a 128-row x kN tile of one head: rows are tokens (M), outputs N.  Both
// operands come by TMA as 128B-swizzled boxes of 64 elements; rows past the last are
// filled with zeros on the way in and dropped on the way out, so that nothing is checked
// in between.  W_k[h] stands [128][512] in memory: for expand its rows are outputs
// (K-major B), for absorb they are the sum's index (MN-major B), and no transposed copy
// is kept.  Accumulators in TMEM, fp32; a warp packs its 32 rows to bf16 (one rounding)
// into swizzled shared memory 64 columns at a time and a TMA store takes them out.
//
// Bound: absorb and project have 85 to 100 flops a byte, so HBM at every size; expand
// 512, so the tensor cores once the rows are many.
#include "pa_common.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;                 // rows of a tile
constexpr int kBox = kRows * 128;          // A of a k-block: 128 rows x 64 bf16
constexpr int kThreads = 192;              // epilogue warps 0-3, TMA warp 4, MMA warp 5

// kind::f16 with bf16 operands, fp32 accumulators
constexpr uint32_t idesc_bf16(uint32_t M, uint32_t N) { return idesc_f16_f32(M, N) | (1u << 7) | (1u << 10); }

template <int kN, int kKBlocks, int kStages>
struct ProductSmem {
  static constexpr int kB = kN * 128;                // B of a k-block
  static constexpr int kStage = kBox + kB;
  static constexpr int kBars = kStages * kStage;     // full[S] empty[S] done
  static constexpr int kMisc = kBars + (2 * kStages + 1) * 8;
  static constexpr int kTotal = kMisc + 16 + 1024;
  static_assert(kN / 64 * kBox <= kBars, "the output is staged where the operands were");
};

struct ProductParams {
  int32_t* status;
  int64_t wait_limit_ns;
  int32_t rows, heads, splits;     // kN-wide pieces of a head's outputs
  int32_t skip_first_load;
  // absorb: the dims copied behind the product
  const __nv_bfloat16* src;
  __nv_bfloat16* dst;
  int64_t src_stride, dst_stride;  // elements a row
};

enum { kAbsorb = 0, kProject = 1, kExpand = 2 };

template <int kOp, int kN, int kKBlocks, int kStages, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas)
    product_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_o2,
                   const ProductParams p) {
  using SM = ProductSmem<kN, kKBlocks, kStages>;
  constexpr bool kBmn = kOp == kAbsorb;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBars);
  uint64_t* empty = full + kStages;
  uint64_t* done = empty + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kMisc);
  volatile int* abort_any = reinterpret_cast<volatile int*>(smem + SM::kMisc + 4);
  const uint32_t s_base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // pieces of a head, then heads, then row blocks: CTAs that run together share rows of x
  const int per_block = p.heads * p.splits;
  const int rb = (int)(blockIdx.x / (uint32_t)per_block), rest = (int)(blockIdx.x % (uint32_t)per_block);
  const int head = rest / p.splits, n0 = rest % p.splits * kN;
  const int row0 = rb * kRows;
  const uint64_t limit = (uint64_t)p.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_any = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(tmem_slot, kN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ================================================================ TMA
    if (lane == 0) {
      tma_prefetch_desc(&tm_x);
      tma_prefetch_desc(&tm_w);
      tma_prefetch_desc(&tm_o);
      int issued = 0;
      for (int kb = 0; kb < kKBlocks; ++kb) {
        const int s = kb % kStages;
        if (kb >= kStages && !wait_or_abort(&empty[s], (kb / kStages - 1) & 1, limit, abort_any)) {
          if (!*abort_any) record_status(p.status, PA_ERR_DEVICE_TIMEOUT, (int)blockIdx.x);
          *abort_any = 1;
          break;
        }
        if (p.skip_first_load && kb == 0 && blockIdx.x == 0) break;   // failure-detection test hook
        uint8_t* st = smem + s * SM::kStage;
        mbar_arrive_expect_tx(&full[s], SM::kStage);
        tma_load_3d(st, &tm_x, &full[s], 64 * kb, kOp == kExpand ? 0 : head, row0);
        if constexpr (kBmn) {
#pragma unroll
          for (int j = 0; j < kN / 64; ++j)
            tma_load_3d(st + kBox + j * 64 * 128, &tm_w, &full[s], n0 + 64 * j, 64 * kb, head);
        } else {
          tma_load_3d(st + kBox, &tm_w, &full[s], 64 * kb, n0, head);
        }
        ++issued;
      }
      // every issued load lands before the CTA exits
      for (int kb = issued > kStages ? issued - kStages : 0; kb < issued; ++kb)
        mbar_wait(&full[kb % kStages], (kb / kStages) & 1, kDrainNs);
    }
  } else if (warp == 5) {
    // ================================================================ MMA
    constexpr uint32_t idesc = idesc_bf16(kRows, kN) | (kBmn ? 1u << 16 : 0u);
    for (int kb = 0; kb < kKBlocks; ++kb) {
      const int s = kb % kStages;
      if (!wait_or_abort(&full[s], (kb / kStages) & 1, limit, abort_any, whole_warp)) {
        if (lane == 0) {
          if (!*abort_any) record_status(p.status, PA_ERR_DEVICE_TIMEOUT, (int)blockIdx.x);
          *abort_any = 1;
          __threadfence_block();
        }
        break;
      }
      tc_fence_after();
      const uint32_t a = s_base + s * SM::kStage, b = a + kBox;
      if (elect_one()) {
#pragma unroll
        for (int kq = 0; kq < 4; ++kq)
          mma_ss(tmem, sdesc_k128(a + 32 * kq),
                 kBmn ? sdesc_mn128(b + kq * 16 * 128, 64 * 128, 1024) : sdesc_k128(b + 32 * kq), idesc,
                 (kb | kq) ? 1u : 0u);
        tc_commit(&empty[s]);
      }
      __syncwarp();
    }
    if (elect_one()) tc_commit(done);   // whatever was issued completes before TMEM is released
    __syncwarp();
    mbar_wait(done, 0, kDrainNs);
  } else {
    // ================================================================ epilogue
    if (kOp == kAbsorb && n0 == 0) {
      // the rotated dims, 8 lanes a row, while the product is made
      const int64_t so = (int64_t)head * 192 + 128 + 8 * (lane & 7), to = (int64_t)head * 576 + 512 + 8 * (lane & 7);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int row = row0 + 32 * warp + 4 * k + (lane >> 3);
        if (row < p.rows)
          *reinterpret_cast<uint4*>(p.dst + row * p.dst_stride + to) =
              __ldg(reinterpret_cast<const uint4*>(p.src + row * p.src_stride + so));
      }
    }
    const bool ok = wait_or_abort(done, 0, limit, abort_any, whole_warp) && !__any_sync(0xffffffffu, *abort_any);
    tc_fence_after();
    const int r0 = row0 + 32 * warp;
    if (ok && r0 < p.rows) {
      const uint32_t t = tmem + ((uint32_t)(32 * warp) << 16);
#pragma unroll 1
      for (int j = 0; j < kN / 64; ++j) {
        // 64 columns of this warp's 32 rows, where the operands were
        const uint32_t box = s_base + j * kBox + warp * 32 * 128, line = box + lane * 128;
        uint32_t v[64];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld16(t + 64 * j + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&v[16 * c]));
        tmem_wait_ld();
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
        if (lane == 0) {
          if (kOp == kExpand && j >= 2) tma_store_3d(&tm_o2, box, 64 * (j - 2), head, r0);
          else tma_store_3d(&tm_o, box, n0 + 64 * j, head, r0);
        }
      }
      if (lane == 0) bulk_store_drain();   // shared memory is read before the CTA leaves
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kN);
}

template <int kOp, int kN, int kKBlocks, int kStages, int kCtas>
cudaError_t launch(const CUtensorMap (&tm)[4], const ProductParams& p, cudaStream_t stream) {
  auto kern = product_kernel<kOp, kN, kKBlocks, kStages, kCtas>;
  constexpr int smem = ProductSmem<kN, kKBlocks, kStages>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = ((int64_t)p.rows + kRows - 1) / kRows * p.heads * p.splits;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  kern<<<(uint32_t)grid, kThreads, smem, stream>>>(tm[0], tm[1], tm[2], tm[3], p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mla_product(const MlaProduct& m, const FaultCfg& fc, cudaStream_t stream) {
  ProductParams p{};
  p.status = m.status;
  p.wait_limit_ns = fc.wait_limit_ns;
  p.skip_first_load = fc.skip_first_load;
  p.rows = m.rows;
  p.heads = m.heads;
  p.src = static_cast<const __nv_bfloat16*>(m.x);
  p.dst = static_cast<__nv_bfloat16*>(m.out);
  p.src_stride = m.x_stride;
  p.dst_stride = m.out_stride;
  switch (m.op) {
    // outputs a tile, stages and CTAs an SM, by the times of 48, 777 and 2048 tokens of 128
    // heads: absorb 256 outputs, 2 CTAs (4.6, 37.2, 82.5 us; 128 outputs, 3 CTAs 39.3 and
    // 88.3 of the longer ones); project 2 stages, 3 CTAs (27.4 and 62.3 of the longer
    // ones; 3 stages, 2 CTAs 29.2 and 64.8; 64 outputs 31.5 and 67.5)
    case kAbsorb:
      p.splits = 2;
      return launch<kAbsorb, 256, 2, 2, 2>(m.tm, p, stream);
    case kProject:
      p.splits = 1;
      return launch<kProject, 128, 8, 2, 3>(m.tm, p, stream);
    default:
      p.splits = 1;
      return launch<kExpand, 256, 8, 4, 1>(m.tm, p, stream);
  }
}

}  // namespace pa
