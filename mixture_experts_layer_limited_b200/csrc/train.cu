// Training GEMMs of the SwiGLU experts and the router on the tensor cores: the
// forward that keeps the pre-activations, and the backward pass.
//
// Forward, per expert segment (rows r, weights w13 = [w1; w3], w2):
//   [g | u] = a w13^T,  h = SiLU(g) * u,  out = row_w * (h w2^T).
// Given d_out (gradient of out) and the saved pre-activations [g | u]:
//   dh0 = d_out w2,  d_row_w[r] = sum_i h[r,i] dh0[r,i],  dh = row_w * dh0,
//   dg = dh * u * s * (1 + g (1 - s)),  du = dh * g * s,   s = sigmoid(g),
//   d_a = [dg | du] w13,  d_w13 = [dg | du]^T a,  d_w2 = d_out^T (row_w * h).
//
// Two kernels:
//  train_gemm_kernel  the products with a weight. As in the forward GEMMs the
//                 weight is the MMA's A operand (M = features) and the
//                 segment's rows are B. In the backward products the weight's
//                 features are its contiguous dimension, so A is MN-major: no
//                 transposed copy of the weights is made. The dh0 form turns
//                 each tile into dg, du and row_w * h in its epilogue, and
//                 leaves the partial sums of d_row_w.
//  wgrad_kernel   the weight gradients: rows are the reduction, both operands
//                 MN-major. A segment's last K block is cut at the segment's
//                 end: rows behind it are zeroed in shared memory in both
//                 operands (a neighbour's row may hold anything, and
//                 0 * NaN is NaN).
#include "segments.cuh"

namespace moe {

constexpr int kChunkBytes = 64 * 128;   // one MN-major TMA box: 64 K rows x 64 features (128 B)

// Shared-memory descriptor of an MN-major operand written by TMA with 128-byte
// swizzle as boxes of 64 K rows x 64 features: boxes of further features are
// kChunkBytes apart (leading dimension), groups of 8 K rows 1024 B apart
// (stride dimension). A K step of 16 starts 2048 B further on.
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kChunkBytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;

// ========================================================================
// CTA pairs
// ========================================================================
// Loads of a CTA of a pair into its own shared memory, completing on a barrier
// of either CTA (`bar`: its address in the cluster).
//
// The TMA unit was the bound of these kernels wherever HBM was not: fitted over
// their variants, a load costs it about 58 cycles and 20.5 more per KB. So every
// operand comes as one box a block, as large as the tile allows, and results
// are stored by the epilogue warps themselves.
__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                                 int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(void* smem_dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                                 int32_t y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
// A 32-bit shared variable of the other CTA.
__device__ __forceinline__ uint32_t ld_cluster(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}

// The CTA-pair forms of the tcgen05 calls.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void umma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on `bar` of both CTAs once every MMA issued so far by this thread is
// done. `lead`: the pair's first CTA in the cluster.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar, int lead = 0) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3 << lead))
      : "memory");
}
// Arrives on the pair's first CTA's copy of `bar`. What the arrival hands over is
// shared memory of this SM that the MMAs read in place: a thread that wrote it
// has made its stores visible to them with fence.proxy.async before, so the
// arrival itself needs no order beyond this CTA's (a release at cluster scope
// waits for a memory barrier of the whole GPU: 870 us instead of 790 for the
// weight gradients of 251 rows on each of 32 experts). The relaxed form is for
// threads that wrote nothing.
__device__ __forceinline__ void mbar_arrive_first(uint64_t* bar, int lead = 0) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(bar), lead))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_first_relaxed(uint64_t* bar, int lead = 0) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(bar), lead))
               : "memory");
}
// Arrives on `bar` of this CTA once every MMA issued so far by this thread is done.
__device__ __forceinline__ void umma_commit_first(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// After an abort one CTA may have loaded into a stage what the other had not
// got to: the first CTA completes the phases both should have filled, arms the
// one only the second started, so that every load has landed before either CTA
// leaves. loads[i]: blocks a CTA has loaded into stage i on the first CTA's
// full[i]; load_bytes[i]: its part of the last one (the same in both CTAs where
// both loaded it). Called by one thread of the first CTA between two cluster
// barriers.
template <int STAGES>
__device__ void pair_drain(uint64_t* full, const uint32_t* loads, const uint32_t* load_bytes, volatile int* abort_flag,
                           const int* abort_word, int lead = 0) {
  if (!*abort_flag && ld_cluster(abort_word, lead + 1) == 0) return;
  for (int i = 0; i < STAGES; ++i) {
    const uint32_t mine = loads[i], theirs = ld_cluster(&loads[i], lead + 1);
    if (mine > theirs)
      asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&full[i])),
                   "r"(load_bytes[i])
                   : "memory");
    else if (theirs > mine)
      mbar_arrive_expect_tx(&full[i], ld_cluster(&load_bytes[i], lead + 1));
    const uint32_t n = mine > theirs ? mine : theirs;
    if (n) mbar_wait_drain(&full[i], (n - 1) & 1u);
  }
}

// ========================================================================
// Products of a segment's rows with a weight
// ========================================================================
// SiLU's sigmoid with the fast exponential and division (relative error about
// 2^-21, below that of the tensor cores' fp32 sums it multiplies).
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// A pair of CTAs shares a tile of SUBS * 256 weight-side rows x up to 256 token
// rows (M = 256 per MMA, N a multiple of 32), 64 of K a block: each CTA loads
// its SUBS * 128 weight-side rows and half of the token rows, and has the
// accumulator rows of its own features for all the tile's token rows.
//   SUBS = 2 (forward, long K): 48 KB loaded per CTA and block for the products
//     a lone CTA's 256 x 256 tile loads 64 KB for; the accumulators fill TMEM,
//     and the four stages loaded meanwhile hide the epilogue.
//   SUBS = 1 (dh0, and d_a-like products of K <= 512): two accumulators, so that
//     the epilogue, which is long beside so few products, overlaps the next
//     tile's MMAs. A long dh0 comes in parts (hidden_parts): the first in one
//     accumulator, each further one in the other, from where the epilogue warps add
//     it to the first (in TMEM); then the next tile begins in the free one.
// Measured on B200, this kernel's dh0 and d_a products at V3 widths, 256 rows
// on each of 32 experts, and at V2-Lite's layer: one CTA per tile of 256 x 256
// with one accumulator 365 / 445 and 374 / 253 us; SUBS = 1 303 / 568 and
// 233 / 317 us (dh0 in one sum; in parts 290 to 360 and 260); SUBS = 2 for d_a
// 480 and 293. The forward at V3 widths: 440 us in a burst of 30 ms (1100
// TFLOP/s), 507 to 600 in a long loop, where the power cap holds the clock near
// 1.2 GHz.
//   forward: sub-tile 0 holds the gate rows of the CTA's 128 features, sub-tile
//   1 their up rows, so that one thread has both.
// Warp 0 loads, warp 1 of the first CTA issues the MMAs, twelve epilogue warps:
// warp w reads TMEM lanes 32 (w % 4).. and every third 32-row chunk.
template <int MODE, int SUBS>
struct PairCfg {
  static constexpr int KB = 64;
  static constexpr int STAGES = SUBS == 2 ? 4 : 6;
  static constexpr uint32_t SUB_BYTES = 2 * kChunkBytes;
  static constexpr uint32_t A_BYTES = SUBS * SUB_BYTES;
  static constexpr uint32_t STAGE_BYTES = A_BYTES + 128 * 128;
  static constexpr int ACCS = SUBS == 2 ? 1 : 2;
  static constexpr int FEATS = MODE == TRAIN_FORWARD ? 256 : SUBS * 256;   // features per tile, half of them per CTA
  static constexpr int EPIW = 12;
  static constexpr int THREADS = 64 + 32 * EPIW;
};
template <int MODE, int SUBS>
struct PairSmem {
  using C = PairCfg<MODE, SUBS>;
  uint8_t stage[C::STAGES][C::STAGE_BYTES];              // 1024-byte aligned
  __nv_bfloat16 tile[C::EPIW][32 * 32];
  uint64_t full_bar[C::STAGES], empty_bar[C::STAGES], tmem_full[2], tmem_empty[2], drain_bar;
  uint32_t tmem_base;
  uint32_t loads[C::STAGES];                             // blocks loaded into a stage
  uint32_t load_bytes[C::STAGES];                        // of the last one, this CTA's part
  int abort_flag;
  SegSched sched;
};

template <int MODE, int SUBS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg<MODE, SUBS>::THREADS, 1)
train_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ HalfMaps tmB, const TrainGemmArgs a) {
  static_assert(MODE != TRAIN_FORWARD || SUBS == 2, "forward: gate and up are the two sub-tiles");
  static_assert(MODE != TRAIN_HIDDEN || SUBS == 1, "dh0: two accumulators");
  using C = PairCfg<MODE, SUBS>;
  constexpr int KB = C::KB, STAGES = C::STAGES, EPIW = C::EPIW, ACCS = C::ACCS;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  PairSmem<MODE, SUBS>& sm = *reinterpret_cast<PairSmem<MODE, SUBS>*>(dsmem);
  if ((smem_u32(dsmem) & 1023u) != 0) {                            // the swizzled tiles need it (the same in both CTAs)
    flag_status(a.status, MOE_DEVSTAT_TIMEOUT);
    return;
  }
  uint64_t *full_bar = sm.full_bar, *empty_bar = sm.empty_bar, *tmem_full = sm.tmem_full, *tmem_empty = sm.tmem_empty;
  volatile int* abort_flag = &sm.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int first = static_cast<int>(cluster_id_x()), stride = static_cast<int>(gridDim.x) / 2;
  const SegProblem sp{a.rows, a.groups, a.offsets, a.n_mblk, 256, 32, a.status};

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
      sm.loads[i] = sm.load_bytes[i] = 0;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tmem_full[i], 1);
      mbar_init(&tmem_empty[i], 2 * EPIW);                         // one arrival per epilogue warp of both CTAs
    }
    mbar_init(&sm.drain_bar, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    for (int i = 0; i < 8; ++i) tma_prefetch_desc(&tmB.box[i]);
  }
  if (warp == 1) tmem_alloc_pair(&sm.tmem_base, 512);
  griddep_wait();
  griddep_launch_dependents();                                     // after the wait: see wgrad_kernel's `after`
  if (warp == 2) build_schedule(sm.sched, sp, lane);
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                                  // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem_base = sm.tmem_base;
  const int total = total_tiles(sm.sched, sp);
  const int nk = (a.K + KB - 1) / KB;
  const int parts = MODE == TRAIN_HIDDEN ? a.parts : 1;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_once = policy_evict_first();
      const uint64_t pol_reuse = policy_evict_normal();
      const uint64_t pol_x = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int group = 0;
      for (int t = first; t < total && ok && !*abort_flag; t += stride) {
        const SegTile ti = decode_tile(sm.sched, sp, t, group);
        const uint64_t pol_w = ti.ntb > 1 ? pol_reuse : pol_once;
        const uint32_t bytes = C::A_BYTES + static_cast<uint32_t>(ti.N) * 64u;   // this CTA's half of a block
        const CUtensorMap* mB = &tmB.box[ti.N / 32 - 1];
        const int brow = ti.row0 + rank * (ti.N / 2);
        const int m0 = ti.mb * C::FEATS + C::FEATS / 2 * rank;      // this CTA's first feature
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, a.status, a.wait_ns)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * bytes);
          ++sm.loads[stage];
          sm.load_bytes[stage] = bytes;
          const uint32_t bar = mapa_shared(smem_u32(&full_bar[stage]), 0);
          // the weight's box of this block (make_train_weight_tmap), and the block in the rows' operand
          int x = 0, y = 0, z = 0, bx = kb * KB;
          if (MODE == TRAIN_FORWARD) {
            if (a.tiled) {
              z = (ti.g * (a.M / 128) + m0 / 128) * nk + kb;
            } else {
              x = kb * KB;
              y = m0;
              z = 2 * ti.g;
            }
          } else if (a.tiled) {
            y = (kb & 3) * 64;
            z = (ti.g * (a.K / 256) + (kb >> 2)) * (a.M / 64) + m0 / 64;
            if (MODE == TRAIN_ROWS)                                 // K runs in the tiled w13's row order
              bx = (kb >> 2) * 128 + (kb & 1) * 64 + ((kb & 2) ? a.K / 2 : 0);
          } else {
            y = ti.g * a.K + kb * KB;
            z = m0 / 64;
          }
          tma_load_3d_pair(sm.stage[stage], &tmA, bar, x, y, z, pol_w);
          tma_load_2d_pair(sm.stage[stage] + C::A_BYTES, mB, bar, bx, brow, pol_x);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // the MMAs' last commits to this CTA's barriers have arrived before it leaves
      for (int i = 0; i < STAGES && ok && !*abort_flag; ++i) {
        ok = mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, a.status, a.wait_ns);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      // as little as possible between the blocks' MMAs (see wgrad_kernel)
      constexpr uint64_t kA = MODE == TRAIN_FORWARD ? 2 : 128, kB = 2;   // descriptor units (16 B) per K step of 16
      const uint64_t ad0 = MODE == TRAIN_FORWARD ? sw128_desc(smem_u32(sm.stage[0])) : mn_desc(smem_u32(sm.stage[0]));
      const uint64_t bd0 = sw128_desc(smem_u32(sm.stage[0]) + C::A_BYTES);
      int st = 0;
      uint32_t phase = 0, freed = 0;                               // freed: parity of each accumulator's next wait
      bool ok = true;
      int group = 0, cur = 0;
      for (int t = first; t < total && ok; t += stride) {
        const SegTile ti = decode_tile(sm.sched, sp, t, group);
        const uint32_t idesc = make_idesc(1u, 256u, static_cast<uint32_t>(ti.N)) | (MODE == TRAIN_FORWARD ? 0u : kIdescAMn);
        const int keep = cur;
        uint32_t d0 = tmem_base + cur * 256;
        ok = mbar_wait(&tmem_empty[cur], ((freed >> cur) & 1u) ^ 1u, abort_flag, a.status, a.wait_ns);
        if (!ok) break;
        freed ^= 1u << cur;
        tc_fence_after();
        uint32_t acc = 0;
        int part = 1, part_end = nk / parts;
        for (int kb = 0; kb < nk; ++kb) {
          if (MODE == TRAIN_HIDDEN && kb == part_end) {            // the next part, in another accumulator
            umma_commit_pair(&tmem_full[cur]);
            part_end = ++part * nk / parts;
            cur = keep ^ 1;
            ok = mbar_wait(&tmem_empty[cur], ((freed >> cur) & 1u) ^ 1u, abort_flag, a.status, a.wait_ns);
            if (!ok) break;
            freed ^= 1u << cur;
            tc_fence_after();
            d0 = tmem_base + cur * 256;
            acc = 0;
          }
          ok = mbar_wait(&full_bar[st], phase, abort_flag, a.status, a.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = ad0 + st * (C::STAGE_BYTES >> 4), bd = bd0 + st * (C::STAGE_BYTES >> 4);
#pragma unroll
          for (int kk = 0; kk < KB / 16; ++kk) {
#pragma unroll
            for (int s = 0; s < SUBS; ++s)
              umma_bf16_pair(d0 + s * 256, ad + s * (C::SUB_BYTES >> 4) + kk * kA, bd + kk * kB, idesc, acc);
            acc = 1;
          }
          umma_commit_pair(&empty_bar[st]);
          if (++st == STAGES) { st = 0; phase ^= 1u; }
        }
        if (ok) umma_commit_pair(&tmem_full[cur]);
        cur = ACCS == 2 ? keep ^ 1 : 0;                            // the next tile's first part
      }
      umma_commit_first(&sm.drain_bar);                            // all issued MMAs must finish before TMEM is released
      mbar_wait_drain(&sm.drain_bar, 0);
    }
  } else {
    const int q = warp & 3, c0 = (warp - 2) / 4;
    constexpr int cstep = EPIW / 4;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    const size_t ld = 2 * static_cast<size_t>(a.M);                // of the pre-activations and their gradients
    __nv_bfloat16* stg = sm.tile[warp - 2];
    uint32_t done = 0;                                             // parity of each accumulator's next wait
    int group = 0, cur = 0;
    for (int t = first; t < total; t += stride) {
      const SegTile ti = decode_tile(sm.sched, sp, t, group);
      const int nchunk = (ti.N + 31) / 32;
      const int keep = cur;
      const uint32_t acc0 = lane_addr + cur * 256;
      const int f0 = ti.mb * C::FEATS + C::FEATS / 2 * rank + 32 * q;
      constexpr int PASSES = MODE == TRAIN_FORWARD ? 1 : SUBS;     // sub-tiles of features
      // the first piece's other inputs, before the wait
      TileRegs gr, ur;
      const bool mine = f0 < a.M && c0 < nchunk;                   // the last tile of a matrix may be part empty
      if (MODE == TRAIN_HIDDEN && mine) {
        gr = load_tile_regs(a.gu, ld, ti.row0 + c0 * 32, ti.n_valid - c0 * 32, f0, lane);
        ur = load_tile_regs(a.gu, ld, ti.row0 + c0 * 32, ti.n_valid - c0 * 32, a.M + f0, lane);
      }
      if (MODE == TRAIN_ROWS && SUBS == 1 && mine && a.add)
        gr = load_tile_regs(a.add, static_cast<size_t>(a.M), ti.row0 + c0 * 32, ti.n_valid - c0 * 32, f0, lane);
      if (!mbar_wait_warp(&tmem_full[cur], (done >> cur) & 1u, abort_flag, a.status, a.wait_ns)) break;
      done ^= 1u << cur;
      cur = ACCS == 2 ? keep ^ 1 : 0;
      tc_fence_after();
      if (MODE == TRAIN_HIDDEN && parts > 1) {
        // each further part is added to the first one's accumulator; its own is then
        // free for another part
        bool ok = true;
        for (int p = 1; p < parts; ++p) {
          ok = mbar_wait_warp(&tmem_full[cur], (done >> cur) & 1u, abort_flag, a.status, a.wait_ns);
          if (!ok) break;
          done ^= 1u << cur;
          tc_fence_after();
          auto free_other = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_first_relaxed(&tmem_empty[cur]);
          };
          if (c0 >= nchunk) free_other();
          for (int c = c0; c < nchunk; c += cstep) {
            float x[32], y[32];
            tmem_ld32(lane_addr + cur * 256 + c * 32, y);
            tmem_ld32(acc0 + c * 32, x);
            tmem_ld_wait();
            if (c + cstep >= nchunk) free_other();
            uint32_t r[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(x[j] + y[j]);
            tmem_st32(acc0 + c * 32, r);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        if (!ok) break;
      }
#pragma unroll 1
      for (int s = 0; s < PASSES; ++s) {
        const int feat0 = f0 + s * 128;
        if (feat0 >= a.M) break;
        const uint32_t acc = acc0 + s * 256;
#pragma unroll 1
        for (int c = c0; c < nchunk; c += cstep) {
          const int row0 = ti.row0 + c * 32, n_rows = ti.n_valid - c * 32;
          const int row1 = row0 + 32 * cstep, n_rows1 = n_rows - 32 * cstep;   // the next chunk's
          float v[32];
          uint32_t p[16];
          tmem_ld_frag(acc + c * 32, v);
          if (MODE == TRAIN_FORWARD) {
            // h from the fp32 sums; the pre-activations are rounded once, for the backward pass
            float u[32];
            tmem_ld_frag(acc + 256 + c * 32, u);
            tmem_ld_wait();
            pack_frag(v, p);
            store_frag(stg, p, lane, a.gu, ld, row0, n_rows, feat0);
            pack_frag(u, p);
            store_frag(stg, p, lane, a.gu, ld, row0, n_rows, a.M + feat0);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = silu(v[j]) * u[j];
            pack_frag(v, p);
            store_frag(stg, p, lane, a.h, static_cast<size_t>(a.M), row0, n_rows, feat0);
          } else if (MODE == TRAIN_HIDDEN) {
            float w[8];
            frag_row_values(a.row_w ? a.row_w + row0 : nullptr, n_rows, lane, 1.0f, w);
            uint32_t g[16], u[16];
            spread_frag(stg, gr, lane, g);
            spread_frag(stg, ur, lane, u);
            if (c + cstep < nchunk) {                              // the next chunk's, while this one is computed
              gr = load_tile_regs(a.gu, ld, row1, n_rows1, feat0, lane);
              ur = load_tile_regs(a.gu, ld, row1, n_rows1, a.M + feat0, lane);
            }
            tmem_ld_wait();
            // g <- dg, u <- du, p <- row_w h; sums of h dh0 over this thread's four features of each row.
            // dg, du and row_w h are computed in fp32 and rounded to bf16 here, once: they are the
            // second products' operands, and those multiply them with bf16 weights and rows (an
            // instruction takes one type). With it the gradients are 2.4e-3 of their norm from the
            // 64-bit value; fp32 throughout and rounded at the end, 1.7e-3.
            float sum[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int i = (k >> 1) & 3;
              const float2 gk = unpack_bf16(g[k]), uk = unpack_bf16(u[k]);
              float dg[2], du[2], hw[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float ge = e ? gk.y : gk.x, ue = e ? uk.y : uk.x, we = w[2 * i + e], dh0 = v[2 * k + e];
                const float sg = sigmoid(ge);
                const float act = ge * sg;                         // SiLU(g)
                const float dh = dh0 * we, h = act * ue;
                sum[2 * i + e] = fmaf(h, dh0, sum[2 * i + e]);
                hw[e] = h * we;
                dg[e] = dh * ue * sg * fmaf(ge, 1.0f - sg, 1.0f);
                du[e] = dh * act;
              }
              g[k] = pack_bf16(dg[0], dg[1]);
              u[k] = pack_bf16(du[0], du[1]);
              p[k] = pack_bf16(hw[0], hw[1]);
            }
            store_frag(stg, g, lane, a.d_gu, ld, row0, n_rows, feat0);
            store_frag(stg, u, lane, a.d_gu, ld, row0, n_rows, a.M + feat0);
            store_frag(stg, p, lane, a.h, static_cast<size_t>(a.M), row0, n_rows, feat0);
            // over the 8 lanes t / 4 that hold the other features: lane t is left with sum t / 4's row
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) {
              const bool up = ((lane >> 2) & d) != 0;
#pragma unroll
              for (int k = 0; k < d; ++k) {
                const float send = up ? sum[k] : sum[k + d], keep = up ? sum[k + d] : sum[k];
                sum[k] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * d);
              }
            }
            const int r = frag_row(lane, lane >> 3, (lane >> 2) & 1);
            if (r < n_rows) a.partial[static_cast<size_t>(feat0 / 32) * a.rows + row0 + r] = sum[0];
          } else {
            tmem_ld_wait();
            if (SUBS == 1 && a.add) {                              // only a short K has rows to add to
              uint32_t add[16];
              spread_frag(stg, gr, lane, add);
              if (c + cstep < nchunk)
                gr = load_tile_regs(a.add, static_cast<size_t>(a.M), row1, n_rows1, feat0, lane);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 o = unpack_bf16(add[k]);
                v[2 * k] += o.x;
                v[2 * k + 1] += o.y;
              }
            }
            pack_frag(v, p);
            store_frag(stg, p, lane, a.out, static_cast<size_t>(a.M), row0, n_rows, feat0);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_first_relaxed(&tmem_empty[keep]);
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                                                  // neither CTA issues anything any more
  if (rank == 0 && threadIdx.x == 0) pair_drain<STAGES>(sm.full_bar, sm.loads, sm.load_bytes, abort_flag, &sm.abort_flag);
  cluster_sync();                                                  // nothing of either CTA is used any more
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// A row's d_row_w: its partial sums, in feature order.
__device__ __forceinline__ float sum_partials(const float* partial, int n, int rows, int r) {
  float s = 0.0f;
#pragma unroll 8
  for (int i = 0; i < n; ++i) s += partial[static_cast<size_t>(i) * rows + r];
  return s;
}
// d_row_w where no weight gradients are asked for (else wgrad_kernel does it);
// rows outside [offsets[0], offsets[groups]) are left as they were.
__global__ void __launch_bounds__(256)
row_w_grad_kernel(int rows, int n, const float* partial, const int32_t* offsets, int groups,
                  float* d_row_w) {
  launch_dependents_if_small();
  griddep_wait();
  const int r = blockIdx.x * 256 + threadIdx.x;
  const int lo = offsets ? offsets[0] : 0, hi = offsets ? offsets[groups] : rows;   // r < rows bounds both
  if (r >= rows || r < lo || r >= hi) return;
  d_row_w[r] = sum_partials(partial, n, rows, r);
}

// ========================================================================
// Weight gradients: C[g] [M, N] = A[rows of g, M]^T B[rows of g, N]
// ========================================================================
// A pair of CTAs (a cluster of two) shares one tile of 256 features of A by 256
// of B (128 where N leaves no more), K = the segment's rows in blocks of 64:
// tcgen05.mma.cta_group::2 with M = 256. Each CTA holds 128 features of A and
// half of B's in shared memory and the accumulator rows of its features in TMEM,
// twice (2 x 256 columns), so that a tile's stores overlap the next tile's
// products. Long segments are bound by the tensor cores under the power cap,
// segments of a few rows by the output's bytes.
//
// Warp 0 loads its CTA's operands (one box each a block); both CTAs' loads
// complete on the first CTA's full_bar, whose warp 1 issues the MMAs for both
// and commits to both. Eight warps take the accumulator to shared memory as
// 128-byte-swizzled boxes of 32 rows and store them with TMA (bf16, or fp32,
// stored or added to what is there). Rows behind the segment's end in its last K
// step are zeroed in both operands by a warp of their own (a neighbour's row may
// hold anything, and 0 * NaN is NaN); that block's loads complete on a barrier of
// each CTA's own.
//
// `after`: the kernel before this one in the stream is a train_gemm_kernel this
// one does not depend on. It let this one start only after all before it had
// completed, so this one runs beside it (on the SMs it leaves) and waits for its
// end before its own.
//
// Measured on B200 at V3 widths, 32 experts: 256 rows each 777 us (3.6 TB/s
// written, 930 TFLOP/s), 251 rows 792 us, 16 rows 470 us (6.0 TB/s written).
// The router's (8192 rows, 256 x 7168: 28 tiles) over 56 pairs: its gradient,
// with dx, 110 us instead of 120.
// What was slower at 256 rows: one CTA per tile of 256 x 256 with one
// accumulator 935 us; the warps storing 16 or 32 bytes a thread themselves 890
// and 970; 128-row store boxes 808; B's blocks kept for a run of eight tiles,
// two fifths of the loads saved, 790: neither loads nor stores alone set the
// pace, and with operands of zeros, which draw less power, 672 us are left.
struct WgradCfg {
  static constexpr int KB = 64;                          // rows per stage
  static constexpr int STAGES = 6;
  static constexpr uint32_t PAIR = 2 * kChunkBytes;      // one load: KB rows x 128 features, as two 64-feature boxes
  static constexpr uint32_t STAGE_BYTES = 2 * PAIR;      // A's, then B's
  static constexpr int EPIW = 8;
  static constexpr int THREADS = 96 + 32 * EPIW;         // loads, MMAs, epilogue, tails
};
// All shared memory of the kernel: the stages take all but a few KB of the
// SM's, so nothing is left for a static allocation beside an aligned dynamic one.
struct WgradSmem {
  using C = WgradCfg;
  uint8_t stage[C::STAGES][C::STAGE_BYTES];              // 1024-byte aligned
  uint8_t out[C::EPIW][32 * 128];                        // one store box per epilogue warp
  uint64_t full_bar[C::STAGES], tail_full[C::STAGES], tail_done[C::STAGES], empty_bar[C::STAGES];
  uint64_t tmem_full[2], tmem_empty[2], drain_bar;
  uint32_t tmem_base;
  uint32_t loads[C::STAGES], tails[C::STAGES];           // blocks loaded into a stage, on full_bar and on tail_full
  uint32_t load_bytes[C::STAGES];
  int abort_flag;
  int off[kMaxGroups + 1];
};

// The tiles of a pair, `stride` apart, in order: problem p, group g, blocks mi
// and ni (fastest) of 256 features of A and B. Steps by adding with carries:
// divisions a tile cost its MMAs a third of their time at 256 rows.
struct WgradIter {
  int t, stride, p, g, mi, ni;
  int step_g, step_m, step_n;                            // stride in this problem's groups, mi and ni
  __device__ __forceinline__ void place(const WgradArgs& a) {
    const bool second = t >= a.prob[0].tiles;
    p = second ? 1 : 0;
    const int local = second ? t - a.prob[0].tiles : t;
    const int per = a.prob[p].per_group, nn = a.prob[p].n_blocks;
    g = local / per;
    mi = (local - g * per) / nn;
    ni = local - g * per - mi * nn;
    step_g = stride / per;
    step_m = (stride - step_g * per) / nn;
    step_n = stride - step_g * per - step_m * nn;
  }
  __device__ __forceinline__ WgradIter(const WgradArgs& a, int first, int stride_) : t(first), stride(stride_) { place(a); }
  __device__ __forceinline__ void next(const WgradArgs& a, int total) {
    t += stride;
    if (t >= total) return;
    if (p == 0 && t >= a.prob[0].tiles) { place(a); return; }
    const int nn = a.prob[p].n_blocks, nm = a.prob[p].m_blocks;
    ni += step_n;
    mi += step_m;
    g += step_g;
    if (ni >= nn) { ni -= nn; ++mi; }
    if (mi >= nm) { mi -= nm; ++g; }
  }
};
struct WgradTile { int p, g, m, n, N, k0, kn; };

// `off`: the segments' starts in shared memory (cut_starts); part `part` of SPLIT
// of the segment's blocks of rows.
template <int SPLIT>
__device__ __forceinline__ WgradTile wgrad_tile(const WgradArgs& a, const int* off, const WgradIter& i, int part) {
  WgradTile w;
  w.p = i.p;
  w.g = i.g;
  w.m = i.mi * 256;
  w.n = i.ni * 256;
  w.N = a.prob[i.p].N;
  w.k0 = off[w.g];
  w.kn = off[w.g + 1] - w.k0;
  if (SPLIT > 1) {
    const int blocks = (w.kn + WgradCfg::KB - 1) / WgradCfg::KB;
    const int from = part * blocks / SPLIT * WgradCfg::KB, to = (part + 1) * blocks / SPLIT * WgradCfg::KB;
    w.kn = max(min(w.kn, to) - from, 0);
    w.k0 += from;
  }
  return w;
}

// Parts that a tile's sum over so many blocks of rows is made in, in turn one
// accumulator's and the other's. The tensor cores cut their sums towards zero every
// 16 rows, always to the same side: sums over 8192 rows came out short by 2.9e-5
// of themselves with equal signs, 9.1e-6 with random ones. fp32 gradients are summed in parts of at most 896
// rows (hidden_parts), joined with rounding in TMEM; in bf16 ones it does not show.
// What the joins cost on B200: one group of 8192 rows at V3 widths 830 -> 838 us of
// the weight gradients' call, a gate's gradient (8192 tokens x 7168, 256 experts)
// 33 -> 36 us.
template <bool F32>
__device__ __forceinline__ int wgrad_parts(int blocks) {
  constexpr int kMost = 896 / WgradCfg::KB;
  return F32 && blocks > kMost ? (blocks + kMost - 1) / kMost : 1;
}

template <int SPLIT, bool F32>
__global__ void __cluster_dims__(2 * SPLIT, 1, 1) __launch_bounds__(WgradCfg::THREADS, 1)
wgrad_kernel(const __grid_constant__ WgradArgs a) {
  using C = WgradCfg;
  constexpr int KB = C::KB, STAGES = C::STAGES, EPIW = C::EPIW;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  WgradSmem& sm = *reinterpret_cast<WgradSmem*>(dsmem);
  if ((smem_u32(dsmem) & 1023u) != 0) {                            // the swizzled tiles need it (the same in both CTAs)
    flag_status(a.status, MOE_DEVSTAT_TIMEOUT);
    return;
  }
  uint64_t *full_bar = sm.full_bar, *empty_bar = sm.empty_bar, *tmem_full = sm.tmem_full, *tmem_empty = sm.tmem_empty;
  const int* off = sm.off;
  volatile int* abort_flag = &sm.abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = static_cast<int>(cluster_ctarank());
  const int rank = crank & 1, lead = crank & ~1, part = crank >> 1;   // in the pair; its first CTA; which pair
  const int first = static_cast<int>(cluster_id_x()), stride = static_cast<int>(gridDim.x) / (2 * SPLIT);
  auto sA = [&](int st) { return sm.stage[st]; };
  auto sB = [&](int st) { return sm.stage[st] + C::PAIR; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&sm.tail_full[i], 1);
      mbar_init(&sm.tail_done[i], 2);                            // both CTAs' tail warps
      mbar_init(&empty_bar[i], 1);
      sm.loads[i] = sm.tails[i] = 0;
      sm.load_bytes[i] = C::STAGE_BYTES;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tmem_full[i], 1);
      mbar_init(&tmem_empty[i], 2 * EPIW);                         // one arrival per epilogue warp of both CTAs
    }
    mbar_init(&sm.drain_bar, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    for (int p = 0; p < a.n_prob; ++p) {
      tma_prefetch_desc(&a.prob[p].tmA);
      tma_prefetch_desc(&a.prob[p].tmB);
      tma_prefetch_desc(&a.prob[p].tmOut);
    }
  }
  if (warp == 1) tmem_alloc_pair(&sm.tmem_base, 512);
  if (!a.after) {
    griddep_wait();
    griddep_launch_dependents();
  }
  bool lie = true;
  for (int i = threadIdx.x; i <= a.groups; i += blockDim.x) {
    sm.off[i] = a.offsets ? a.offsets[i] : i * a.rows;
    lie = lie && (i == a.groups || !a.offsets || seg_lies(sm.off[i], a.offsets[i + 1], a.rows));
  }
  tc_fence_before();
  if (!__syncthreads_and(lie)) {
    if (warp == 2) cut_starts(sm.off, a.offsets, a.groups, a.rows, a.status, lane);
    __syncthreads();
  }
  cluster_sync();                                                  // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem_base = sm.tmem_base;
  const int total = a.prob[0].tiles + (a.n_prob > 1 ? a.prob[1].tiles : 0);

  // 32 features x `cols` columns from c of tile w, one feature a lane, through this warp's box
  auto store = [&](const WgradTile& w, int c, const float (&v)[32], const float (&v2)[32]) {
    uint8_t* box = sm.out[warp - 2];                               // 32 rows x 128 B
    // the last store of this box has been read
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
    uint8_t* row = box + lane * 128;
    if (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float4*>(row + ((i ^ (lane & 7)) << 4)) =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float* f = i < 4 ? v + 8 * i : v2 + 8 * (i - 4);
        uint4 u;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
        *reinterpret_cast<uint4*>(row + ((i ^ (lane & 7)) << 4)) = u;
      }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      const WgradProblem& pr = a.prob[w.p];
      const int y = w.g * pr.M + w.m + 128 * rank + 32 * (warp & 3);
      if (a.accumulate)
        asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];"
                     ::"l"(reinterpret_cast<uint64_t>(&pr.tmOut)), "r"(smem_u32(box)), "r"(w.n + c), "r"(y)
                     : "memory");
      else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
                     ::"l"(reinterpret_cast<uint64_t>(&pr.tmOut)), "r"(smem_u32(box)), "r"(w.n + c), "r"(y)
                     : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  };
  const int cols = F32 ? 32 : 64;                                // columns of a box

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (WgradIter i(a, first, stride); i.t < total && ok && !*abort_flag; i.next(a, total)) {
        const WgradTile w = wgrad_tile<SPLIT>(a, off, i, part);
        const WgradProblem& pr = a.prob[w.p];
        const int m = w.m + 128 * rank;
        const int nb = w.n / 64 + (w.N - w.n > 128 ? 2 : 1) * rank;    // this CTA's half of B's features
        for (int k = 0; k < w.kn; k += KB) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, a.status, a.wait_ns)) { ok = false; break; }
          const bool tail = w.kn - k <= KB && (w.kn & 15);         // rows to zero
          uint32_t bar;
          if (tail) {
            mbar_arrive_expect_tx(&sm.tail_full[stage], C::STAGE_BYTES);
            bar = mapa_shared(smem_u32(&sm.tail_full[stage]), crank);
            ++sm.tails[stage];
          } else {
            if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * C::STAGE_BYTES);
            bar = mapa_shared(smem_u32(&full_bar[stage]), lead);
            ++sm.loads[stage];
          }
          if (pr.a_flat) {                                         // rows not a whole number of boxes wide
            tma_load_2d_pair(sA(stage), &pr.tmA, bar, m, w.k0 + k, pol);
            tma_load_2d_pair(sA(stage) + kChunkBytes, &pr.tmA, bar, m + 64, w.k0 + k, pol);
          } else {
            tma_load_3d_pair(sA(stage), &pr.tmA, bar, 0, w.k0 + k, m / 64, pol);
          }
          tma_load_3d_pair(sB(stage), &pr.tmB, bar, 0, w.k0 + k, nb, pol);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // the MMAs' last commits to this CTA's barriers have arrived before it leaves
      for (int i = 0; i < STAGES && ok && !*abort_flag; ++i) {
        ok = mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, a.status, a.wait_ns);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (*abort_flag)                                             // this CTA's tail loads; the others: pair_drain
        for (int i = 0; i < STAGES; ++i)
          if (sm.tails[i]) mbar_wait_drain(&sm.tail_full[i], (sm.tails[i] - 1) & 1u);
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      // Nothing but the wait stands between one block's MMAs and the next's:
      // their issue keeps only a few queued, and 700 cycles of bookkeeping a
      // block (512 of MMAs) cost a third of the rate.
      const uint64_t ad0 = mn_desc(smem_u32(sm.stage[0]));         // descriptor of stage 0's A
      int st = 0, cur = 0;                                         // stage; the next part's accumulator
      uint32_t full_par = 0, tail_par = 0, freed = 0;              // parity of each stage's or accumulator's next wait
      bool ok = true;
      for (WgradIter i(a, first, stride); i.t < total && ok; i.next(a, total)) {
        const WgradTile w = wgrad_tile<SPLIT>(a, off, i, part);
        const uint32_t idesc = make_idesc(1u, 256u, w.N - w.n > 128 ? 256u : 128u) | kIdescAMn | kIdescBMn;
        const int even = w.kn / KB, rest = w.kn - even * KB;       // blocks of 64 rows, and the last one's rows
        const int blocks = even + (rest > 0), parts = wgrad_parts<F32>(blocks), keep = cur;
        for (int p = 1, kb = 0; p <= parts; ++p) {                 // the first part in one accumulator, further ones in the other
          ok = mbar_wait(&tmem_empty[cur], ((freed >> cur) & 1u) ^ 1u, abort_flag, a.status, a.wait_ns);
          if (!ok) break;
          freed ^= 1u << cur;
          tc_fence_after();
          const uint32_t d0 = tmem_base + cur * 256;
          const int end = p < parts ? p * blocks / parts : even;
          uint32_t acc = 0;
          for (; kb < end; ++kb) {
            ok = mbar_wait(&full_bar[st], (full_par >> st) & 1u, abort_flag, a.status, a.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = ad0 + st * (C::STAGE_BYTES >> 4), bd = ad + (C::PAIR >> 4);
#pragma unroll
            for (int kk = 0; kk < KB / 16; ++kk) {                 // 2048 B a step, in the descriptors' 16-byte units
              umma_bf16_pair(d0, ad + kk * 128, bd + kk * 128, idesc, acc);
              acc = 1;
            }
            umma_commit_pair(&empty_bar[st], lead);
            full_par ^= 1u << st;
            if (++st == STAGES) st = 0;
          }
          if (ok && p == parts && rest > 0) {
            if (rest & 15) {
              ok = mbar_wait(&sm.tail_done[st], (tail_par >> st) & 1u, abort_flag, a.status, a.wait_ns);
              tail_par ^= 1u << st;
            } else {
              ok = mbar_wait(&full_bar[st], (full_par >> st) & 1u, abort_flag, a.status, a.wait_ns);
              full_par ^= 1u << st;
            }
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = ad0 + st * (C::STAGE_BYTES >> 4), bd = ad + (C::PAIR >> 4);
            for (int kk = 0; kk < (rest + 15) / 16; ++kk) {
              umma_bf16_pair(d0, ad + kk * 128, bd + kk * 128, idesc, acc);
              acc = 1;
            }
            umma_commit_pair(&empty_bar[st], lead);
            if (++st == STAGES) st = 0;
          }
          if (!ok) break;
          umma_commit_pair(&tmem_full[cur], lead);
          cur = keep ^ 1;
        }
      }
      // all issued MMAs must finish before TMEM is released
      umma_commit_first(&sm.drain_bar);
      mbar_wait_drain(&sm.drain_bar, 0);
    }
  } else if (warp == 2 + EPIW) {
    // rows behind the segment's end in the last block: zeroed as soon as they land
    int stage = 0;
    uint32_t par = 0;
    for (WgradIter i(a, first, stride); i.t < total; i.next(a, total)) {
      const WgradTile w = wgrad_tile<SPLIT>(a, off, i, part);
      const int blocks = (w.kn + KB - 1) / KB;
      if (w.kn & 15) {
        const int st = (stage + blocks - 1) % STAGES;
        const int valid = w.kn - (blocks - 1) * KB;
        if (!mbar_wait_warp(&sm.tail_full[st], (par >> st) & 1u, abort_flag, a.status, a.wait_ns)) break;
        par ^= 1u << st;
        const int nz = ((valid + 15) / 16 * 16 - valid) * 128;     // bytes per box: A's two boxes, then B's
        uint8_t* base = sA(st) + valid * 128;
        for (int i = lane * 16; i < nz; i += 512)
#pragma unroll
          for (int b = 0; b < 4; ++b) *reinterpret_cast<uint4*>(base + b * kChunkBytes + i) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive_first(&sm.tail_done[st], lead);
      }
      stage = (stage + blocks) % STAGES;
    }
  } else {
    const int q = warp & 3, half = (warp - 2) / 4;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    // d_row_w, while the first tile's products run: rows outside [offsets[0],
    // offsets[groups]) are left as they were
    if (a.d_row_w) {
      const int hi = off[a.groups];
      for (int r = off[0] + blockIdx.x * 32 * EPIW + threadIdx.x - 64; r < hi; r += gridDim.x * 32 * EPIW)
        a.d_row_w[r] = sum_partials(a.partial, a.n_partial, a.rows, r);
    }
    int cur = 0;
    uint32_t done = 0;                                             // parity of each accumulator's next wait
    for (WgradIter i(a, first, stride); i.t < total; i.next(a, total)) {
      const WgradTile w = wgrad_tile<SPLIT>(a, off, i, part);
      const WgradProblem& pr = a.prob[w.p];
      const int width = w.N - w.n > 128 ? 256 : 128;
      const int m = w.m + 128 * rank + 32 * q;                     // this warp's 32 features of A
      const int keep = cur;
      const uint32_t acc = lane_addr + keep * 256;
      if (!mbar_wait_warp(&tmem_full[keep], (done >> keep) & 1u, abort_flag, a.status, a.wait_ns)) break;
      done ^= 1u << keep;
      cur = keep ^ 1;
      tc_fence_after();
      // each further part is read, its accumulator handed back, and added to the first's
      bool ok = true;
      for (int p = wgrad_parts<F32>((w.kn + KB - 1) / KB); p > 1; --p) {
        ok = mbar_wait_warp(&tmem_full[cur], (done >> cur) & 1u, abort_flag, a.status, a.wait_ns);
        if (!ok) break;
        done ^= 1u << cur;
        tc_fence_after();
#pragma unroll 1
        for (int c = 32 * half; c < width; c += 64) {              // this warp's columns
          float x[32], y[32];
          tmem_ld32(lane_addr + cur * 256 + c, y);
          tmem_ld32(acc + c, x);
          tmem_ld_wait();
          if (c + 64 >= width) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_first_relaxed(&tmem_empty[cur], lead);
          }
          uint32_t r[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(x[j] + y[j]);
          tmem_st32(acc + c, r);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
      if (!ok) break;
      if (SPLIT > 1) continue;                                     // one tile, summed over its pairs below
      const bool empty = w.kn == 0;
      // adding nothing needs no store, and rows past the matrix have none
      if (!(empty && a.accumulate) && m < pr.M) {
#pragma unroll 1
        for (int c = half * cols; c < width; c += 2 * cols) {
          float v[32], v2[32];
          if (!empty) {
            tmem_ld32(acc + c, v);
            if (!F32) tmem_ld32(acc + c + 32, v2);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = v2[j] = 0.0f;
          }
          store(w, c, v, v2);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_first_relaxed(&tmem_empty[keep], lead);
    }
    if (SPLIT == 1 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                                                  // no CTA of the cluster issues anything any more
  if constexpr (SPLIT > 1) {
    // Pair j gets the others' sums of its 256 / SPLIT columns in the stages, by
    // now free: [other pair][column][128 features], adds them in that order and stores.
    constexpr int CW = 256 / SPLIT;
    const bool epi = warp >= 2 && warp < 2 + EPIW;
    const int q = warp & 3, half = (warp - 2) / 4;
    const uint32_t acc = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    float* got = reinterpret_cast<float*>(sm.stage[0]);
    const WgradIter i(a, first, stride);
    const WgradTile w = wgrad_tile<SPLIT>(a, off, i, part);
    tc_fence_after();
    if (epi) {
      for (int d = 1; d < SPLIT; ++d) {
        const int to = (part + d) % SPLIT, slot = part < to ? part : part - 1;
        const uint32_t dst = mapa_shared(smem_u32(got + (slot * CW) * 128 + 32 * q + lane), 2 * to + rank);
        for (int c = 32 * half; c < CW; c += 64) {
          float v[32];
          tmem_ld32(acc + to * CW + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + (c + j) * 512), "f"(w.kn ? v[j] : 0.0f) : "memory");
        }
      }
    }
    cluster_sync();
    const int m = w.m + 128 * rank + 32 * q;
    if (epi && !*abort_flag && m < a.prob[w.p].M) {
      for (int c = half * cols; c < CW; c += 2 * cols) {
        float v[32], v2[32];
        tmem_ld32(acc + part * CW + c, v);
        if (!F32) tmem_ld32(acc + part * CW + c + 32, v2);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (!w.kn) v[j] = 0.0f;
          if (!w.kn || F32) v2[j] = 0.0f;
          for (int o = 0; o < SPLIT - 1; ++o) {
            const float* f = got + (o * CW + c + j) * 128 + 32 * q + lane;
            v[j] += f[0];
            if (!F32) v2[j] += f[32 * 128];
          }
        }
        store(w, part * CW + c, v, v2);
      }
      if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) pair_drain<STAGES>(sm.full_bar, sm.loads, sm.load_bytes, abort_flag, &sm.abort_flag, lead);
  cluster_sync();                                                  // nothing of either CTA is used any more
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
  if (a.after) griddep_wait();                                     // what follows this kernel follows that one too
}

// ========================================================================
// Router: d_logits from the gradients of the routing weights
// ========================================================================
// w_j = scale * s_j (/ sum_i s_i if normalised), s the softmax or sigmoid
// scores of the k chosen experts (the selection itself has no gradient):
//   sigmoid: d_logit_j = scale dw_j s_j (1 - s_j);
//   softmax: d_logit_e = p_e (ds_e - sum_i p_i ds_i), ds = scale dw, 0 for experts
//     not chosen;
//   normalised, with the shares r_j = s_j / S:  scale r_j (dw_j - sum_i dw_i r_i),
//     for sigmoid times 1 - s_j; the other experts' are 0.
// The shares come from scores scaled by e^-m, m the largest chosen logit (no more
// than 0 for sigmoid), so that they are finite where the scores themselves leave
// fp32's range (logits below -87). The bf16 copy of d_logits is for the gate's
// products, whose operands are of one type: one rounding more for dx and d_gate
// (2.3e-3 of their norm from the 64-bit value instead of 1.7e-3), none for the fp32
// d_logits. One warp per token: lane j holds slot j, lane l
// the experts l, l + 32, ... . Bound by its E logits' bytes: 8192 tokens x 256
// experts (21 MB, from L2 in part) in 5.5 to 6.8 us as a graph.
__global__ void __launch_bounds__(256)
route_backward_kernel(int T, int E, int k, int scoring, int norm, float scale, const float* logits,
                      const int32_t* ids, const float* d_w,
                      const int32_t* slot_to_row, float* d_logits,
                      __nv_bfloat16* d_logits16, int32_t* status) {
  constexpr int PER = 8;                                           // E <= 256
  launch_dependents_if_small();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= T) return;
  const float* lg = logits + static_cast<size_t>(t) * E;
  int id = -1;
  float dw = 0.0f, l_id = 0.0f;
  if (lane < k) {
    const size_t slot = static_cast<size_t>(t) * k + lane;
    id = ids[slot];
    if (id >= E) { flag_status(status, MOE_DEVSTAT_BAD_EXPERT_ID); id = -1; }
    if (id >= 0) {
      long long at = slot;
      if (slot_to_row) at = slot_to_row[slot];
      if (at >= 0 && at < static_cast<long long>(T) * k) dw = d_w[at];
      else flag_status(status, MOE_DEVSTAT_BAD_EXPERT_ID);
      l_id = lg[id];
    }
  }
  auto all_sum = [](float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
  };
  auto all_max = [](float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
  };
  // each slot's part of its expert's gradient, but for the sum over all experts
  // that a softmax which is not renormalised adds
  const bool full = scoring == MOE_SOFTMAX && !norm;
  float p[PER];                                                    // full: this lane's probabilities
  float part, dot = 0.0f;
  if (full) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      p[i] = e < E ? lg[e] : -INFINITY;
      top = fmaxf(top, p[i]);
    }
    top = all_max(top);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      p[i] = expf(p[i] - top);
      sum += p[i];
    }
    const float inv = 1.0f / all_sum(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] *= inv;
    part = id < 0 ? 0.0f : scale * dw;
    dot = all_sum(id < 0 ? 0.0f : part * (expf(l_id - top) * inv));
  } else if (norm) {
    const bool sig = scoring == MOE_SIGMOID;
    float m = all_max(id < 0 ? -INFINITY : l_id);
    if (sig) m = fminf(m, 0.0f);
    // sigmoid, with t = e^-|l|: s is 1 / (1 + t) above 0 and e^l / (1 + t) below,
    // 1 - s is t / (1 + t) and 1 / (1 + t): neither cancels
    const float t = sig ? expf(-fabsf(l_id)) : 0.0f, inv = 1.0f / (1.0f + t);
    const bool up = sig && l_id > 0.0f;
    const float q = id < 0 ? 0.0f : up ? inv : expf(l_id - m) * inv;
    const float sum = all_sum(q), r = id < 0 ? 0.0f : q / sum;
    const float mean = all_sum(dw * r);
    part = id < 0 ? 0.0f : scale * r * (dw - mean);
    if (sig) part *= up ? t * inv : inv;
  } else {
    const float s = 1.0f / (1.0f + expf(-l_id));
    part = id < 0 ? 0.0f : scale * dw * (s * (1.0f / (1.0f + expf(l_id))));
  }
  float out[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) out[i] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int idj = __shfl_sync(0xffffffffu, id, j);
    const float partj = __shfl_sync(0xffffffffu, part, j);
#pragma unroll
    for (int i = 0; i < PER; ++i) out[i] += idj == lane + 32 * i ? partj : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    if (e < E) {
      const float d = full ? p[i] * (out[i] - dot) : out[i];
      d_logits[static_cast<size_t>(t) * E + e] = d;
      if (d_logits16) d_logits16[static_cast<size_t>(t) * E + e] = __float2bfloat16_rn(d);
    }
  }
}

// ------------------------------------------------------------------------
// host-side launch helpers (called from api.cu)
// ------------------------------------------------------------------------
template <int MODE, int SUBS>
static cudaError_t train_gemm(const CUtensorMap& tmA, const HalfMaps& tmB, TrainGemmArgs a, int num_sms,
                              cudaStream_t stream) {
  using C = PairCfg<MODE, SUBS>;
  constexpr size_t smem = sizeof(PairSmem<MODE, SUBS>);
  static_assert(smem <= 232448, "train_gemm_kernel's shared memory exceeds an SM's");
  cudaError_t e = cudaFuncSetAttribute(train_gemm_kernel<MODE, SUBS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  a.n_mblk = (a.M + C::FEATS - 1) / C::FEATS;
  a.parts = MODE == TRAIN_HIDDEN ? hidden_parts(a.K) : 1;
  const long long most = train_tiles(a.rows, a.groups, a.M, C::FEATS);
  const int pairs = num_sms / 2 < most ? num_sms / 2 : static_cast<int>(most);
  return launch_after(train_gemm_kernel<MODE, SUBS>, 2 * pairs, C::THREADS, smem, stream, tmA, tmB, a);
}
cudaError_t launch_train_gemm(int mode, int subs, const CUtensorMap& tmA, const HalfMaps& tmB, const TrainGemmArgs& a,
                              int num_sms, cudaStream_t stream) {
  return mode == TRAIN_FORWARD  ? train_gemm<TRAIN_FORWARD, 2>(tmA, tmB, a, num_sms, stream)
         : mode == TRAIN_HIDDEN ? train_gemm<TRAIN_HIDDEN, 1>(tmA, tmB, a, num_sms, stream)
         : subs == 2            ? train_gemm<TRAIN_ROWS, 2>(tmA, tmB, a, num_sms, stream)
                                : train_gemm<TRAIN_ROWS, 1>(tmA, tmB, a, num_sms, stream);
}

cudaError_t launch_row_w_grad(int rows, int n, const float* partial, const int32_t* offsets, int groups, float* d_row_w,
                              cudaStream_t stream) {
  return launch_after(row_w_grad_kernel, (rows + 255) / 256, 256, 0, stream, rows, n, partial, offsets, groups, d_row_w);
}

cudaError_t launch_route_backward(int T, int E, int k, int scoring, int norm, float scale, const float* logits,
                                  const int32_t* ids, const float* d_w, const int32_t* slot_to_row, float* d_logits,
                                  void* d_logits16, int32_t* status, cudaStream_t stream) {
  return launch_after(route_backward_kernel, (T + 7) / 8, 256, 0, stream, T, E, k, scoring, norm, scale, logits, ids, d_w,
                      slot_to_row, d_logits, static_cast<__nv_bfloat16*>(d_logits16), status);
}

template <int SPLIT, bool F32>
static cudaError_t wgrad(const WgradArgs& a, int clusters, cudaStream_t stream) {
  constexpr size_t smem = sizeof(WgradSmem);
  static_assert(smem <= 232448, "wgrad_kernel's shared memory exceeds an SM's");
  cudaError_t e = cudaFuncSetAttribute(wgrad_kernel<SPLIT, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_after(wgrad_kernel<SPLIT, F32>, 2 * SPLIT * clusters, WgradCfg::THREADS, smem, stream, a);
}
template <bool F32>
static cudaError_t wgrad_any(const WgradArgs& a, int num_sms, cudaStream_t stream) {
  int tiles = 0;
  bool wide = true;                                    // whole tiles of 256 columns
  for (int p = 0; p < a.n_prob; ++p) {
    tiles += a.prob[p].tiles;
    wide = wide && a.prob[p].N % 256 == 0;
  }
  // where the kernel before leaves most SMs idle, this one takes those alone: a
  // pair that had to wait for that one's end would do its share of the tiles late
  const int all = num_sms / 2, room = a.after && 2 * a.beside <= all ? all - a.beside : all;
  // Few tiles of many rows (the router's): each split over two or four pairs, as
  // long as all have room at once (148 SMs take 33 clusters of four CTAs or 15 of
  // eight: 16 tiles of 2048 rows in two turns of the latter 25 us) and 256 rows a
  // pair and segment.
  const int rows = a.rows / a.groups;
  if (wide && 4 * tiles <= room && tiles <= num_sms * 15 / 148 && rows >= 4 * 256) return wgrad<4, F32>(a, tiles, stream);
  if (wide && 2 * tiles <= room && tiles <= num_sms * 33 / 148 && rows >= 2 * 256) return wgrad<2, F32>(a, tiles, stream);
  return wgrad<1, F32>(a, room < tiles ? room : tiles, stream);
}
cudaError_t launch_wgrad(const WgradArgs& a, int num_sms, cudaStream_t stream) {
  return a.f32 ? wgrad_any<true>(a, num_sms, stream) : wgrad_any<false>(a, num_sms, stream);
}

}  // namespace moe
