// pa_mla_prefill.cu - attention of new tokens to expanded latent rows, bf16, tcgen05 + TMA,
// sm_103a: keys of 128 dims a head and 64 rotated ones that all heads share, values of 128.
//
//   s_ij = sm_scale (<q_i[0:128], k_j> + <q_i[128:192], k_rope_j>), out_i = sum_j softmax(s_i)_j v_j
//
// One pass over the keys with a running maximum m and sum l of each row (a row's O is
// rescaled only when its maximum rises by more than 2^8, which leaves 2^(s - m) exact
// for the final division by l).
//
//   * An item is 256 query tokens of one head, two tiles A and B of 128 rows, against a
//     range of positions in steps of 128.  TMEM: S_A 0, S_B 128, O_A 256, O_B 384; P
//     (bf16) takes the place of S and is the A operand of O += P V.
//   * A warp per tile issues its MMAs, PV_X(i) then S_X(i+1): while the softmax of one tile
//     runs, the tensor cores have the other's.  MMAs of one thread execute in order, so
//     S_X(i+1) needs no wait for the PV_X(i) that reads P from its columns, and a finished
//     S_X(i+1) means that O_X holds PV_X(i).  The order runs on over item boundaries; an
//     item's epilogue overlaps the next one's first S.  (What bounded the kernel with one
//     warp for both tiles was that warp: 4060 cycles a step.)
//   * K, V arrive in units of 16 KB through one ring of eight: three of K (128 positions x
//     64 dims, the third from the shared rotated rows) and two of V (64 positions x 128
//     dims, an MN-major B operand as it stands).  With Q (two tiles x 192 dims, 96 KB) that
//     fills shared memory.
//   * Causal: tile A leaves out the step that only B's rows see.
//   * Rows of V past the range are zeroed in shared memory before their MMA (they belong to
//     other sequences and may hold anything; 0 times NaN is NaN), scores by a select.
// Rounding: P to bf16 (V's type; the MMA takes one type), at most 2^-8 p|v| a position,
// rows to bf16, partial rows of split ranges in fp32.
// Bound: the tensor cores, 640 flops per visible (query head, position); 38 heads of 2048 tokens
// against 8192 rows in 236 us, 1730 TFLOP/s, 8192 tokens of 32 heads, causal, 1670.  A step of both
// tiles takes 3150 cycles, its MMAs 2560; the rest is the chain S -> softmax -> PV of each tile.
#include "pa_common.cuh"

namespace pa {
namespace {

constexpr int kTile = 128;                      // positions of a step
constexpr int kUnit = 16384;                    // bytes of a ring slot
constexpr int kSlots = 8;
constexpr int kQTile = 3 * kUnit;               // Q of a tile: three blocks of 64 dims
constexpr int kThreads = 384;                   // softmax A 0-3, softmax B 4-7, TMA 8, MMA A 9, MMA B 10
// registers: 168 a thread at launch, moved to the softmax, whose threads hold a row of scores
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * 168, "the shares add up to the launch's registers");
constexpr int kWarpTma = 8;
constexpr int kWarpMma = 9;
constexpr uint32_t kTmemCols = 512;
constexpr float kTau = 8.0f;                    // lazy-rescale threshold (log2 units)

struct Smem {
  static constexpr int kQ = 0;                          // [A, B][3][128 rows][128 B]
  static constexpr int kRing = 2 * kQTile;
  static constexpr int kBars = kRing + kSlots * kUnit;  // kfull kfree vfull vfree qfull qfree sfull pready[2] odone drain, [2] each
  static constexpr int kMisc = kBars + 22 * 8;
  static constexpr int kTotal = kMisc + 16 + 1024;
  static_assert(kTotal <= 232448, "shared memory overflow");
};

constexpr uint32_t idesc_bf16(uint32_t M, uint32_t N) { return idesc_f16_f32(M, N) | (1u << 7) | (1u << 10); }

// A work item and the steps of its two tiles.
struct Work {
  Item m;        // m.b: row of the sequence's first position
  int nt[2];     // steps of tile A, B
  int n;         // steps of the item
};

__device__ __forceinline__ Work work_of(const int4 a, const int4 c) {
  Work w;
  w.m = item4_from<kTile>(a, c);
  w.n = w.m.ntiles;
  const int lim_a = min(w.m.kv1, w.m.cbase + min(w.m.ntok, 128));   // positions that A's rows see
  w.nt[1] = w.m.ntok > 128 ? w.n : 0;
  w.nt[0] = w.nt[1] ? max(1, (lim_a - w.m.kv0 + kTile - 1) / kTile) : w.n;   // (a split range may hold none of them)
  return w;
}

// (a, b) * c + d in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 c, float2 d) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&c)), "l"(*reinterpret_cast<uint64_t*>(&d)));
  return *reinterpret_cast<float2*>(&r);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}

// Four pieces of 8 words a lane: lane j of a quad goes from pieces 0 .. 3 of its row to
// piece j of the quad's rows 0 .. 3.
__device__ __forceinline__ void quad_transpose(uint32_t (&u)[32], int lane) {
#pragma unroll
  for (int b = 1; b <= 2; b <<= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & b) continue;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        uint32_t &lo = u[8 * i + w], &hi = u[8 * (i + b) + w];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, b);
        lo = up ? got : lo;
        hi = up ? hi : got;
      }
    }
  }
}

// 64 scores -> 2^(s c - m) as bf16 pairs, and their sum before that rounding
__device__ __forceinline__ float exp_half(const uint32_t* v, float c, float neg_m, uint32_t (&o)[32]) {
  const float2 c2 = make_float2(c, c), m2 = make_float2(neg_m, neg_m);
  float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    float2 t = fma2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), c2, m2);
    t.x = fast_exp2(t.x);
    t.y = fast_exp2(t.y);
    sum[e & 1] = add2(sum[e & 1], t);
    __nv_bfloat162 b2 = __floats2bfloat162_rn(t.x, t.y);
    o[e] = *reinterpret_cast<uint32_t*>(&b2);
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v,
                       const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using SM = Smem;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + SM::kBars);   // [step & 1], as the next three
  uint64_t* vfull = kfull + 2;
  uint64_t* kfree = vfull + 2;
  uint64_t* vfree = kfree + 2;
  uint64_t* qfull = vfree + 2;        // [tile], as the next four
  uint64_t* qfree = qfull + 2;
  uint64_t* sfull = qfree + 2;
  uint64_t* pready = sfull + 2;   // [tile][half of the step's positions]
  uint64_t* odone = pready + 4;
  uint64_t* drain = odone + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kMisc);
  volatile int* abort_any = reinterpret_cast<volatile int*>(smem + SM::kMisc + 4);
  volatile int* s_done = reinterpret_cast<volatile int*>(smem + SM::kMisc + 8);   // S steps of tile A that are there
  const uint32_t s_base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int begin = p.work_indptr[blockIdx.x], end = p.work_indptr[blockIdx.x + 1];
  const uint64_t limit = (uint64_t)p.wait_limit_ns;
  const int4* recs = reinterpret_cast<const int4*>(p.items);
  auto work_at = [&](int it) { return work_of(__ldg(recs + 2 * (int64_t)it), __ldg(recs + 2 * (int64_t)it + 1)); };
  auto raise = [&](int it) {
    if (!*abort_any) record_status(p.status, PA_ERR_DEVICE_TIMEOUT, it);
    *abort_any = 1;
  };

  PA_DEBUG_PROLOGUE(smem, SM::kTotal - 1024, p, begin, end);
  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&kfull[x], 1);
      mbar_init(&vfull[x], 1);
      mbar_init(&kfree[x], 2);   // a release by each tile
      mbar_init(&vfree[x], 2);
      mbar_init(&qfull[x], 1);
      mbar_init(&qfree[x], 1);
      mbar_init(&sfull[x], 1);
      mbar_init(&pready[2 * x], 4);
      mbar_init(&pready[2 * x + 1], 4);
      mbar_init(&odone[x], 1);
      mbar_init(&drain[x], 1);
    }
    *abort_any = 0;
    *s_done = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PA_DEBUG_POISON_TMEM(tmem, kTmemCols, warp);

  // one instruction for all warps of a warpgroup
  if (warp >= 8) {
  regs_down<kRegsOther>();
  if (warp == kWarpTma) {
    // ================================================================ TMA
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_r);
      tma_prefetch_desc(&tm_v);
      uint32_t g = 0, nk = 0, nv = 0, nq[2] = {0, 0};   // steps; K, V groups and query tiles begun
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity, int it) {
        if (wait_or_abort(bar, parity, limit, abort_any)) return true;
        raise(it);
        return ok = false;
      };
      auto load_q = [&](int x, const Work& w, int it) {
        if (nq[x] > 0 && !wait(&qfree[x], (nq[x] - 1) & 1, it)) return;
        mbar_arrive_expect_tx(&qfull[x], kQTile);
        for (int d = 0; d < 3; ++d)
          tma_load_3d(smem + SM::kQ + x * kQTile + d * kUnit, &tm_q, &qfull[x], 64 * d, w.m.kvh, w.m.tok0 + 128 * x);
        ++nq[x];
      };
      auto slot = [&](uint32_t u) { return smem + SM::kRing + u % kSlots * kUnit; };
      // Unit u takes the slot of unit u - 8: the third of K(g - 2), both of V(g - 2) and the
      // first two of K(g - 1) for the five units of step g, in this order.
      Work next{};            // read an item ahead
      if (begin < end) next = work_at(begin);
      bool q_there = false;   // tile A's query of the item
      for (int it = begin; it < end && ok; ++it) {
        const Work w = next;
        if (it + 1 < end) next = work_at(it + 1);
        if (!q_there) load_q(0, w, it);
        q_there = false;
        for (int i = 0; i < w.n && ok; ++i, ++g) {
          const int row = w.m.b + w.m.kv0 + i * kTile;
          const uint32_t par2 = ((g - 2) >> 1) & 1;
          if (g >= 2 && !wait(&kfree[g & 1], par2, it)) break;
          if (p.skip_first_load && g == 0) {   // failure-detection test hook
            ok = false;
            break;
          }
          uint64_t* bar = &kfull[g & 1];
          mbar_arrive_expect_tx(bar, 3 * kUnit);
          ++nk;
          tma_load_3d(slot(5 * g), &tm_k, bar, 0, w.m.kvh, row);
          if (g >= 2) wait(&vfree[g & 1], par2, it);   // (loaded all the same: its bytes are announced)
          tma_load_3d(slot(5 * g + 1), &tm_k, bar, 64, w.m.kvh, row);
          tma_load_3d(slot(5 * g + 2), &tm_r, bar, 0, 0, row);
          if (ok && i == 0 && w.nt[1] > 0) load_q(1, w, it);
          // the next item's query as soon as the last S that reads this one's is done (tile A
          // ends a step ahead), before the wait for V's slots
          if (ok && i + 1 == w.n && it + 1 < end && mbar_test_wait(&qfree[0], (nq[0] - 1) & 1)) {
            load_q(0, next, it + 1);
            q_there = true;
          }
          if (!ok || (g >= 1 && !wait(&kfree[(g - 1) & 1], ((g - 1) >> 1) & 1, it))) break;
          bar = &vfull[g & 1];
          mbar_arrive_expect_tx(bar, 2 * kUnit);
          ++nv;
          for (uint32_t h = 0; h < 2; ++h) {
            uint8_t* dst = slot(5 * g + 3 + h);
            tma_load_3d(dst, &tm_v, bar, 0, w.m.kvh, row + 64 * (int)h);
            tma_load_3d(dst + kUnit / 2, &tm_v, bar, 64, w.m.kvh, row + 64 * (int)h);
          }
        }
      }
      // every issued load lands before the CTA exits
      for (uint32_t k = nk > 2 ? nk - 2 : 0; k < nk; ++k) mbar_wait(&kfull[k & 1], (k >> 1) & 1, kDrainNs);
      for (uint32_t k = nv > 2 ? nv - 2 : 0; k < nv; ++k) mbar_wait(&vfull[k & 1], (k >> 1) & 1, kDrainNs);
      for (int x = 0; x < 2; ++x)
        if (nq[x] > 0) mbar_wait(&qfull[x], (nq[x] - 1) & 1, kDrainNs);
    }
  } else if (warp == kWarpMma || warp == kWarpMma + 1) {
    // ================================================================ MMA issue, a warp per tile
    // the whole warp runs the loop (warp-uniform operands)
    constexpr uint32_t idesc_s = idesc_bf16(128, kTile), idesc_pv = idesc_bf16(128, 128) | (1u << 16);
    const int x = warp - kWarpMma;
    const uint32_t ring = s_base + SM::kRing, s_tm = tmem + 128 * x, o_tm = tmem + 256 + 128 * x;
    const uint64_t q = sdesc_k128(s_base + SM::kQ + x * kQTile);
    uint32_t np = 0, nq = 0;   // PV steps and items of this tile
    // One lane issues everything (MMAs of one thread execute in order, its commits cover them),
    // if its own waits have come true.  Each lane waits for itself, and a wait that ran out is its
    // own affair up to the vote behind the step's S, which all branches on `ok` follow.  (A vote
    // in every wait, between P or S and the MMA behind it: one CTA of 400 steps 686 us of 665.)
    const bool leader = elect_one();
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && wait_or_abort(bar, parity, limit, abort_any);
      tc_fence_after();
    };
    // S of step g; first / last step of the item's.  All MMAs of a product leave in one
    // elected branch.
    auto issue_s = [&](uint32_t g, bool first, bool last) {
      if (first) wait(&qfull[x], nq++ & 1);
      wait(&kfull[g & 1], (g >> 1) & 1);
      if (leader && ok) {
#pragma unroll
        for (uint32_t d = 0; d < 3; ++d) {
          const uint64_t k = sdesc_k128(ring + (5 * g + d) % kSlots * kUnit);
#pragma unroll
          for (int kq = 0; kq < 4; ++kq)
            mma_ss(s_tm, q + ((d * kUnit + 32 * kq) >> 4), k + ((32 * kq) >> 4), idesc_s, (d | kq) ? 1u : 0u);
        }
        tc_commit(&sfull[x]);
        tc_commit(&kfree[g & 1]);
        if (last) tc_commit(&qfree[x]);
      }
      ok = warp_all(ok);
    };
    auto issue_pv = [&](uint32_t g, int nvalid, bool first, bool last) {
      wait(&vfull[g & 1], (g >> 1) & 1);
      if (nvalid < kTile) {
        // rows past the range: zero, 8 chunks of 16 bytes a row and block (both tiles' warps
        // do so, each before its own MMAs)
        for (int r = ok ? 8 * nvalid + lane : 8 * kTile; r < 8 * kTile; r += 32) {
          const uint32_t v = ring + (5 * g + 3 + (r >> 9)) % kSlots * kUnit + 16 * (r & 511);
          st_shared_v4(v, make_uint4(0, 0, 0, 0));
          st_shared_v4(v + kUnit / 2, make_uint4(0, 0, 0, 0));
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        wait(&pready[2 * x + h], np & 1);
        const uint64_t v = sdesc_mn128(ring + (5 * g + 3 + h) % kSlots * kUnit, kUnit / 2, 1024);
        if (leader && ok) {
#pragma unroll
          for (int kq = 0; kq < 4; ++kq)
            mma_ts(o_tm, s_tm + 32 * h + 8 * kq, v + ((2048 * kq) >> 4), idesc_pv, (!first || h > 0 || kq > 0) ? 1u : 0u);
          if (h == 1) {
            tc_commit(&vfree[g & 1]);
            if (last) tc_commit(&odone[x]);
          }
        }
        __syncwarp();
      }
      ++np;
    };
    // S runs one step ahead of PV; the step whose PV is due:
    uint32_t due_g = 0, g = 0;
    int due_valid = 0;
    bool due = false, due_first = false, due_last = false;
    int s_of_a = 0;   // S steps of tile A up to this one
    auto flush = [&]() {
      if (due) issue_pv(due_g, due_valid, due_first, due_last);
      due = false;
    };
    Work nxt{};
    if (begin < end) nxt = work_at(begin);
    for (int it = begin; it < end && ok; ++it) {
      const Work w = nxt;
      if (it + 1 < end) nxt = work_at(it + 1);
      const int steps = x ? w.nt[1] : w.nt[0];
      for (int i = 0; i < w.n && ok; ++i, ++g) {
        s_of_a += i < w.nt[0];
        if (i < steps) {
          flush();
          if (x == 1 && i < w.nt[0]) {
            // Tile B's S of a step behind A's: left to themselves the two warps' MMAs share the
            // tensor cores in step, both softmaxes wait for them, and then they for both (38
            // heads of 2048 tokens and 8192 rows 262 us, so 237; taking turns at PV and S both
            // was slower).  A pace, not a dependence: a count, as a barrier's parity could be
            // missed.
            const uint64_t t0 = globaltimer();
            while (ok && *s_done < s_of_a) ok = !*abort_any && globaltimer() - t0 <= limit;
          }
          issue_s(g, i == 0, i + 1 == steps);
          due = true;
          due_g = g;
          due_valid = w.m.kv1 - (w.m.kv0 + i * kTile);
          due_first = i == 0;
          due_last = i + 1 == steps;
        } else {
          // the step is the other tile's alone: its operands are free as far as this one goes
          flush();
          wait(&kfull[g & 1], (g >> 1) & 1);
          if (ok && lane == 0) mbar_arrive(&kfree[g & 1]);
          wait(&vfull[g & 1], (g >> 1) & 1);
          if (ok && lane == 0) mbar_arrive(&vfree[g & 1]);
          ok = warp_all(ok);
        }
      }
      if (!ok && lane == 0) raise(it);
    }
    if (ok) flush();
    ok = warp_all(ok);
    if (!ok && lane == 0) raise(end - 1);
    // drain: every MMA this warp issued completes before TMEM is released
    if (leader) tc_commit(&drain[x]);
    __syncwarp();
    mbar_wait(&drain[x], 0, kDrainNs);
  }
  // (the remaining warps have no role but to complete the warpgroup)
  } else {
    // ================================================================ softmax, thread = row
    regs_up<kRegsSoftmax>();
    const int x = warp >> 2, rr = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lanes + 128 * x, o_tm = tmem + lanes + 256 + 128 * x;
    const float c_log2 = p.sm_scale_log2;
    uint32_t n = 0, items = 0;   // steps, items of this tile
    bool fail = false;
    const int r = 128 * x + rr;
    for (int it = begin; it < end && !fail; ++it) {
      int steps, seen;   // this tile's; positions that the row sees from the step's first on
      {
        const Work w = work_at(it);
        steps = x ? w.nt[1] : w.nt[0];
        seen = min(w.m.kv1, w.m.cbase + r + 1) - w.m.kv0;
      }
      if (it + 1 < end) prefetch_l1(recs + 2 * (int64_t)(it + 1));
      if (steps == 0) continue;   // the item has no rows for this tile
      float m_run = -INFINITY, l = 0.0f;
      for (int i = 0; i < steps; ++i, ++n) {
        if (!wait_or_abort(&sfull[x], n & 1, limit, abort_any, whole_warp)) {
          raise(it);
          fail = true;
          break;
        }
        tc_fence_after();
        if (tid == 0) *s_done = (int)n + 1;
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_tm + 32 * c, v + 32 * c);
        tmem_wait_ld();
        if (seen < kTile) {
#pragma unroll
          for (int e = 0; e < 128; ++e) v[e] = e < seen ? v[e] : 0xFF800000u;   // -inf
        }
        seen -= kTile;
        // the first half's P against the maximum so far, while the step's maximum is taken
        uint32_t o[32];
        float neg_m = m_run == -INFINITY ? 0.0f : -m_run;
        float sum = exp_half(v, c_log2, neg_m, o);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(v[e + k])), __uint_as_float(v[e + k + 4]));
        }
        const float m_tile = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c_log2;
        const bool need = m_tile > m_run + kTau;
        if (__any_sync(0xffffffffu, need)) {
          float alpha = 1.0f;
          if (need) {
            alpha = m_run == -INFINITY ? 0.0f : fast_exp2(m_run - m_tile);
            l *= alpha;
            m_run = m_tile;
          }
          if (i > 0) {   // O holds the PV of the item's earlier steps (they came before this S)
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t t[16];
              tmem_ld16(o_tm + 16 * c, t);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) t[e] = __float_as_uint(__uint_as_float(t[e]) * alpha);
              tmem_st16(o_tm + 16 * c, t);
            }
          }
          neg_m = m_run == -INFINITY ? 0.0f : -m_run;
          sum = exp_half(v, c_log2, neg_m, o);
        }
        // P = 2^(s c - m), bf16, over the first half of S's columns; its halves are announced
        // one by one
        l += sum;
        tmem_st32(s_tm, o);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&pready[2 * x], lane);
        l += exp_half(v + 64, c_log2, neg_m, o);
        tmem_st32(s_tm + 32, o);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&pready[2 * x + 1], lane);
      }
      if (fail) break;
      // ---- epilogue: O / l (the record again, so that nothing of it lives through the steps)
      const Item m = work_at(it).m;
      if (!wait_or_abort(&odone[x], items & 1, limit, abort_any, whole_warp)) {
        raise(it);
        break;
      }
      ++items;
      tc_fence_after();
      const float inv_l = l > 0.0f ? __frcp_rn(l) : 0.0f;
      const bool row_ok = r < m.ntok, final_row = m.nch == 1;
      const int token = m.tok0 + r;
      const int64_t row = final_row ? (int64_t)token * p.q_heads + m.kvh
                                    : ((int64_t)m.chunk + (int64_t)r * m.nch) * p.q_heads + m.kvh;
      if (p.plain_out || !final_row) {
        // Rows without an output epilogue: quads of lanes exchange 32-byte pieces, so that a
        // store instruction writes 8 whole lines (32 sectors of 32 rows each took 4500 cycles
        // a tile, with what the next loads waited behind them)
        const int64_t step = final_row ? p.q_heads : (int64_t)m.nch * p.q_heads;   // rows apart
        const int r4 = r & ~3;
        const int64_t row4 = row - (r - r4) * step;
        if (final_row) {
          uint8_t* dst = reinterpret_cast<uint8_t*>(p.out + row4 * 128) + 32 * (lane & 3);
#pragma unroll 1   // (code that runs once an item: its fetch is what it costs)
          for (int c = 0; c < 2; ++c) {
            uint32_t o[64], u[32];
            tmem_ld32(o_tm + 64 * c, o);
            tmem_ld32(o_tm + 64 * c + 32, o + 32);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[2 * k]) * inv_l, __uint_as_float(o[2 * k + 1]) * inv_l);
              u[k] = *reinterpret_cast<uint32_t*>(&b2);
            }
            quad_transpose(u, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (r4 + k < m.ntok) st_global_32(dst + k * step * 256 + 128 * c, u + 8 * k);
          }
        } else {
          uint8_t* dst = reinterpret_cast<uint8_t*>(reinterpret_cast<float*>(p.part_o) + row4 * 128) + 32 * (lane & 3);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t u[32];
            tmem_ld32(o_tm + 32 * c, u);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * inv_l);
            quad_transpose(u, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (r4 + k < m.ntok) st_global_32(dst + k * step * 512 + 128 * c, u + 8 * k);
          }
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[16];
          tmem_ld16(o_tm + 16 * c, o);
          tmem_wait_ld();
          if (row_ok) {
            float a[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) a[e] = __uint_as_float(o[e]) * inv_l;
            ep_store16(p.ep, p.out, row * 128 + 16 * c, m.kvh * 128 + 16 * c, a);
          }
        }
      }
      tc_fence_before();   // (the next item's first P, behind which its PV writes O, is announced after this)
      if (row_ok) {
        const float ln2 = 0.69314718055994530942f;
        if (final_row) {
          if (p.lse != nullptr) p.lse[row] = l > 0.0f ? (m_run + __log2f(l)) * ln2 : -INFINITY;
        } else {
          p.part_m[row] = l > 0.0f ? m_run * ln2 : -INFINITY;
          p.part_d[row] = l;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();   // the merge grid may be scheduled while the last CTAs finish
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

cudaError_t launch_mla_prefill(const Plan& plan, const AttnParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_r, const CUtensorMap& tm_v, cudaStream_t stream) {
  const cudaError_t e =
      cudaFuncSetAttribute(mla_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::kTotal);
  if (e != cudaSuccess) return e;
  mla_prefill_kernel<<<plan.num_ctas, kThreads, Smem::kTotal, stream>>>(tm_q, tm_k, tm_r, tm_v, p);
  return cudaGetLastError();
}

}  // namespace pa
