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

// The full-precision exponential: d_row_w is an fp32 output, and __expf's
// error would be the largest in it.
__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

// ========================================================================
// Products of a segment's rows with a weight
// ========================================================================
// Sums v[j] (j = 0..31, one value per lane each) over the warp's lanes; lane j
// receives the sum of v[j]. Halving exchange: 31 shuffles instead of 160.
__device__ __forceinline__ float lane_sums(float (&v)[32], int lane) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const bool up = (lane & d) != 0;
#pragma unroll
    for (int j = 0; j < d; ++j) {
      const float send = up ? v[j] : v[j + d];
      const float keep = up ? v[j + d] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, d);
    }
  }
  return v[0];
}

// 32 rows x 32 features of a bf16 matrix through the warp's shared tile:
// v[j] = row j's value of this lane's feature (0 for rows >= n_rows).
struct TileRegs { uint4 r[4]; };
__device__ __forceinline__ TileRegs load_tile_regs(const __nv_bfloat16* src, size_t ld, int row0, int n_rows, int feat0,
                                                   int lane) {
  TileRegs t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (lane >> 2) + 8 * i;
    t.r[i] = r < n_rows ? *reinterpret_cast<const uint4*>(src + static_cast<size_t>(row0 + r) * ld + feat0 + (lane & 3) * 8)
                        : make_uint4(0u, 0u, 0u, 0u);
  }
  return t;
}
__device__ __forceinline__ void spread_tile(__nv_bfloat16* stage, const TileRegs& t, int lane, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(stage + ((lane >> 2) + 8 * i) * 32 + (lane & 3) * 8) = t.r[i];
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __bfloat162float(stage[j * 32 + lane]);
  __syncwarp();
}

// Warp roles and tiling as the forward's grouped GEMM: 256 weight-side rows
// (two 128-row sub-tiles: features f.. and f + 128.., or, forward, the gate and
// up rows of 128 features) x up to 256 token rows per tile, one accumulator
// pair in TMEM, three 64-K stages, EPIW epilogue warps.
template <int MODE, int EPIW>
__global__ void __launch_bounds__(64 + 32 * EPIW, 1)
train_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ TokenMaps tmB, const TrainGemmArgs a) {
  constexpr int STAGES = 3, KB = 64;
  constexpr uint32_t A_SUB_BYTES = 2 * kChunkBytes;
  constexpr uint32_t STAGE_BYTES = 2 * A_SUB_BYTES + 256 * 128;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  __shared__ SegSched sched;
  __shared__ __align__(16) __nv_bfloat16 stage_out[EPIW][32 * 32];
  __shared__ uint64_t full_bar[STAGES], empty_bar[STAGES];
  __shared__ uint64_t tmem_full, tmem_empty, drain_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int issued_parity[STAGES];
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  auto sA = [&](int st) { return smem + st * STAGE_BYTES; };
  auto sB = [&](int st) { return smem + st * STAGE_BYTES + 2 * A_SUB_BYTES; };

  const SegProblem ga{a.rows, a.groups, a.offsets, a.n_mblk, 256, a.status};

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
      issued_parity[i] = -1;
    }
    mbar_init(&tmem_full, 1);
    mbar_init(&tmem_empty, 32 * EPIW);
    mbar_init(&drain_bar, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    for (int i = 0; i < kTokBoxes; ++i) tma_prefetch_desc(&tmB.box[i]);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_s, 512);
    tmem_relinquish();
  }
  if (warp == 2) build_schedule(sched, ga, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_s;
  const int total = sched.tile_start[a.groups];
  const int nk = (a.K + KB - 1) / KB;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_once = policy_evict_first();
      const uint64_t pol_reuse = policy_evict_normal();
      const uint64_t pol_x = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      for (int t = blockIdx.x; t < total && !abort_flag; t += gridDim.x) {
        const SegTile ti = decode_tile(sched, ga, t);
        const int m0 = ti.mb * 256;
        const int nch = MODE == TRAIN_FORWARD ? 4 : min(4, (a.M - m0 + 63) / 64);   // 8 KB pieces of A
        const uint64_t pol_w = ti.ntb > 1 ? pol_reuse : pol_once;
        const uint32_t bytes = static_cast<uint32_t>(nch) * kChunkBytes + static_cast<uint32_t>(ti.N) * 128u;
        bool ok = true;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_flag, a.status, a.wait_ns)) { ok = false; break; }
          mbar_arrive_expect_tx(&full_bar[stage], bytes);
          int bx = kb * KB;                                         // this K block in the rows' operand
          if (MODE == TRAIN_FORWARD) {
            if (a.tiled) {                                          // gate rows, then up rows: one block
              tma_load_2d(sA(stage), &tmA, &full_bar[stage], 0, ((ti.g * a.n_mblk + ti.mb) * nk + kb) * 256, pol_w);
            } else {
              const int y = ti.g * 2 * a.M + ti.mb * 128;
              tma_load_2d(sA(stage), &tmA, &full_bar[stage], kb * KB, y, pol_w);
              tma_load_2d(sA(stage) + A_SUB_BYTES, &tmA, &full_bar[stage], kb * KB, y + a.M, pol_w);
            }
          } else {
            if (MODE == TRAIN_ROWS && a.tiled) {                    // K runs in the tiled w13's row order
              const int sub = kb & 3;
              bx = (kb >> 2) * 128 + (sub & 1) * 64 + (sub >= 2 ? a.K / 2 : 0);
            }
            for (int j = 0; j < nch; ++j) {
              int x = m0 + 64 * j, y = ti.g * a.K + kb * KB;
              if (a.tiled) {                                        // the block of 256 K rows x 64 features, its rows of kb
                y = ((ti.g * (a.K / 256) + (kb >> 2)) * (a.M / 64) + x / 64) * 256 + (kb & 3) * 64;
                x = 0;
              }
              tma_load_2d(sA(stage) + j * kChunkBytes, &tmA, &full_bar[stage], x, y, pol_w);
            }
          }
          uint8_t* bdst = sB(stage);
          uint64_t* fb = &full_bar[stage];
          load_token_rows(ti.N, [&](int which, int off) {
            tma_load_2d(bdst + off * 128, &tmB.box[which], fb, bx, ti.row0 + off, pol_x);
          });
          issued_parity[stage] = static_cast<int>(phase);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
      }
      if (abort_flag) {   // let every issued copy land before the CTA exits
        for (int i = 0; i < STAGES; ++i)
          if (issued_parity[i] >= 0) mbar_wait_drain(&full_bar[i], static_cast<uint32_t>(issued_parity[i]));
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, it = 0;
      for (int t = blockIdx.x; t < total && !abort_flag; t += gridDim.x, ++it) {
        const SegTile ti = decode_tile(sched, ga, t);
        const bool two = MODE == TRAIN_FORWARD || a.M - ti.mb * 256 > 128;
        const uint32_t idesc = make_idesc(1u, 128u, static_cast<uint32_t>(ti.N)) | (MODE == TRAIN_FORWARD ? 0u : kIdescAMn);
        if (!mbar_wait(&tmem_empty, (it & 1u) ^ 1u, &abort_flag, a.status, a.wait_ns)) break;
        tc_fence_after();
        bool ok = true;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&full_bar[stage], phase, &abort_flag, a.status, a.wait_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA(stage)), b0 = smem_u32(sB(stage));
#pragma unroll
          for (int kk = 0; kk < KB / 16; ++kk) {
            const uint32_t acc = (kb | kk) != 0;
            const uint64_t bd = sw128_desc(b0 + kk * 32);
            const uint64_t ad = MODE == TRAIN_FORWARD ? sw128_desc(a0 + kk * 32) : mn_desc(a0 + kk * 2048);
            const uint64_t ad1 = MODE == TRAIN_FORWARD ? sw128_desc(a0 + A_SUB_BYTES + kk * 32)
                                                       : mn_desc(a0 + A_SUB_BYTES + kk * 2048);
            umma_bf16(tmem_base, ad, bd, idesc, acc);
            if (two) umma_bf16(tmem_base + 256, ad1, bd, idesc, acc);
          }
          umma_commit(&empty_bar[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        umma_commit(&tmem_full);
      }
      umma_commit(&drain_bar);   // all issued MMAs must finish before TMEM is released
      mbar_wait_drain(&drain_bar, 0);
    }
  } else {
    const int q = warp & 3;
    constexpr int cstep = EPIW / 4;
    const int c0 = (warp - 2) / 4;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    __nv_bfloat16* stg = stage_out[warp - 2];
    uint32_t it = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x, ++it) {
      const SegTile ti = decode_tile(sched, ga, t);
      const int nchunk = (ti.N + 31) / 32;
      const int nsub = MODE != TRAIN_FORWARD && a.M - ti.mb * 256 > 128 ? 2 : 1;
      // this warp's pieces of 32 features x 32 rows: sub-tile s (forward: both at once), chunk c
      const int per = c0 < nchunk ? (nchunk - c0 + cstep - 1) / cstep : 0;
      const int pieces = nsub * per;
      TileRegs gr, ur;
      if (MODE == TRAIN_HIDDEN && pieces > 0) {                                   // the first piece's pre-activations, before the wait
        const int f = ti.mb * 256 + 32 * q, r = c0 * 32;
        gr = load_tile_regs(a.gu, 2 * static_cast<size_t>(a.M), ti.row0 + r, ti.n_valid - r, f, lane);
        ur = load_tile_regs(a.gu, 2 * static_cast<size_t>(a.M), ti.row0 + r, ti.n_valid - r, a.M + f, lane);
      }
      if (!mbar_wait(&tmem_full, it & 1u, &abort_flag, a.status, a.wait_ns)) break;
      tc_fence_after();
#pragma unroll 1
      for (int p = 0; p < pieces; ++p) {
        const int s = p / per, c = c0 + (p - s * per) * cstep;
        const int feat0 = MODE == TRAIN_FORWARD ? ti.mb * 128 + 32 * q : ti.mb * 256 + s * 128 + 32 * q;
        const int row0 = ti.row0 + c * 32, n_rows = ti.n_valid - c * 32;
        float v[32];
        tmem_ld32(lane_addr + s * 256 + c * 32, v);
        if (MODE == TRAIN_FORWARD) {
          // h from the fp32 sums; the pre-activations are rounded once, for the backward pass
          float u[32];
          tmem_ld32(lane_addr + 256 + c * 32, u);
          tmem_ld_wait();
          const size_t ld = 2 * static_cast<size_t>(a.M);
          store_tile<32>(stg, v, lane, a.gu, ld, row0, n_rows, feat0);
          store_tile<32>(stg, u, lane, a.gu, ld, row0, n_rows, a.M + feat0);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = silu(v[j]) * u[j];
          store_tile<32>(stg, v, lane, a.h, static_cast<size_t>(a.M), row0, n_rows, feat0);
          continue;
        }
        tmem_ld_wait();
        if (MODE == TRAIN_HIDDEN) {
          const size_t ld = 2 * static_cast<size_t>(a.M);
          const float w = (lane < n_rows) ? (a.row_w ? __ldg(a.row_w + row0 + lane) : 1.0f) : 0.0f;
          float g[32], u[32];
          spread_tile(stg, gr, lane, g);
          spread_tile(stg, ur, lane, u);
          if (p + 1 < pieces) {                                     // the next piece's, while this one is computed
            const int s2 = (p + 1) / per, c2 = c0 + (p + 1 - s2 * per) * cstep;
            const int f2 = ti.mb * 256 + s2 * 128 + 32 * q;
            gr = load_tile_regs(a.gu, ld, ti.row0 + c2 * 32, ti.n_valid - c2 * 32, f2, lane);
            ur = load_tile_regs(a.gu, ld, ti.row0 + c2 * 32, ti.n_valid - c2 * 32, a.M + f2, lane);
          }
          // g <- dg, u <- du, v <- h dh0 / row_w * h: one value at a time
          float hw[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            const float sg = sigmoid(g[j]);
            const float act = g[j] * sg;                            // SiLU(g)
            const float dh = v[j] * wj;
            const float h = act * u[j];
            v[j] *= h;
            hw[j] = h * wj;
            const float dg = dh * u[j] * sg * fmaf(g[j], 1.0f - sg, 1.0f);
            u[j] = dh * act;
            g[j] = dg;
          }
          store_tile<32>(stg, g, lane, a.d_gu, ld, row0, n_rows, feat0);
          store_tile<32>(stg, u, lane, a.d_gu, ld, row0, n_rows, a.M + feat0);
          store_tile<32>(stg, hw, lane, a.h, static_cast<size_t>(a.M), row0, n_rows, feat0);
          const float part = lane_sums(v, lane);
          if (lane < n_rows) a.partial[static_cast<size_t>(feat0 / 32) * a.rows + row0 + lane] = part;
        } else {
          if (a.add) {
            float add[32];
            const TileRegs ar = load_tile_regs(a.add, static_cast<size_t>(a.M), row0, n_rows, feat0, lane);
            spread_tile(stg, ar, lane, add);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += add[j];
          }
          store_tile<32>(stg, v, lane, a.out, static_cast<size_t>(a.M), row0, n_rows, feat0);
        }
      }
      tc_fence_before();
      mbar_arrive(&tmem_empty);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, 512);
}

// d_row_w[r] = sum of the row's partial sums, in feature order; rows outside
// [offsets[0], offsets[groups]) are left as they were.
__global__ void __launch_bounds__(256)
row_w_grad_kernel(int rows, int n, const float* __restrict__ partial, const int32_t* __restrict__ offsets, int groups,
                  float* __restrict__ d_row_w) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  const int lo = offsets ? offsets[0] : 0, hi = offsets ? offsets[groups] : rows;   // r < rows bounds both
  if (r >= rows || r < lo || r >= hi) return;
  float s = 0.0f;
  for (int i = 0; i < n; ++i) s += partial[static_cast<size_t>(i) * rows + r];
  d_row_w[r] = s;
}

// ========================================================================
// Weight gradients: C[g] [M, N] = A[rows of g, M]^T B[rows of g, N]
// ========================================================================
// A pair of CTAs (a cluster of two) shares one tile of 256 features of A by 256
// of B (128 where N leaves no more), K = the segment's rows in blocks of 64:
// tcgen05.mma.cta_group::2 with M = 256. Each CTA holds 128 features of A and
// half of B's in shared memory and the accumulator rows of its 128 features in
// TMEM. A CTA so loads 32 KB per block for the products a lone CTA would load
// 48 KB for, and the accumulator takes 256 of the 512 TMEM columns: two of them,
// so a tile's epilogue overlaps the next tile's products. Both count: where a
// segment has few rows the output's bytes bound the work, else the operands'
// way from L2 does. Measured on B200 (V3 widths, 32 experts): one CTA per tile
// of 128 x 256 with two accumulators 933 us at 256 rows per expert and 2815 us
// at 1024; 256 x 256 with one accumulator 935 and 2523 us.
//
// Warp 0 loads its CTA's operands (64 rows x 128 features a load); both CTAs'
// loads complete on the first CTA's full_bar, whose warp 1 issues the MMAs for
// both and commits to both. A last block with rows behind the segment's end in
// its last step goes another way: each CTA's loads complete on a barrier of its
// own, its last warp zeroes those rows and arrives on the first CTA's
// tail_done. (With such a handshake for every block, or the zeroing on the MMA
// warp, its latency set the pace: 251 rows per expert cost 1.5 times what 256
// do.) Eight warps take the accumulator to shared memory as 128-byte-swizzled
// boxes and store them with TMA (bf16, or fp32 added to what is there).
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
  uint8_t out[C::EPIW][32 * 128];
  uint64_t full_bar[C::STAGES], tail_full[C::STAGES], tail_done[C::STAGES], empty_bar[C::STAGES];
  uint64_t tmem_full[2], tmem_empty[2], drain_bar;
  uint32_t tmem_base;
  uint32_t loads[C::STAGES], tails[C::STAGES];           // loads issued into a stage, on full_bar and on tail_full
  int abort_flag;
  int off[kMaxGroups + 1];
};

// Loads of a CTA of a pair into its own shared memory, completing on a barrier
// of either CTA (`bar`: its address in the cluster). 3-D: one box of a matrix
// seen as [N / 64] column blocks of [rows, 64]: 64 rows of two column blocks,
// each block's rows contiguous in shared memory.
__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map, uint32_t bar, int32_t row,
                                                 int32_t block, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row), "r"(block), "l"(policy)
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
// Arrives on `bar` of both CTAs once every MMA issued so far by this thread is done.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// Arrives on the first CTA's copy of `bar` (release at cluster scope); relaxed
// where the thread has written nothing that is read after the barrier.
__device__ __forceinline__ void mbar_arrive_first(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(bar), 0))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_first_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(bar), 0))
               : "memory");
}

struct WgradTile { int p, g, m, n, k0, kn; };

// `off`: the segments' starts in shared memory, cut to the rows there are.
__device__ __forceinline__ WgradTile wgrad_tile(const WgradArgs& a, const int* off, int t) {
  WgradTile w;
  w.p = a.n_prob > 1 && t >= a.prob[0].tiles ? 1 : 0;
  if (w.p) t -= a.prob[0].tiles;
  const WgradProblem& pr = a.prob[w.p];
  w.g = t / pr.per_group;
  const int r = t - w.g * pr.per_group;
  const int mi = r / pr.n_blocks;
  w.m = mi * 256;
  w.n = (r - mi * pr.n_blocks) * 256;
  w.k0 = off[w.g];
  w.kn = off[w.g + 1] - w.k0;
  return w;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(WgradCfg::THREADS, 1)
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
  const int rank = static_cast<int>(cluster_ctarank());
  const int first = static_cast<int>(cluster_id_x()), stride = static_cast<int>(gridDim.x) / 2;
  for (int i = threadIdx.x; i <= a.groups; i += blockDim.x)
    sm.off[i] = a.offsets ? min(max(a.offsets[i], 0), a.rows) : i * a.rows;
  auto sA = [&](int st) { return sm.stage[st]; };
  auto sB = [&](int st) { return sm.stage[st] + C::PAIR; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&sm.tail_full[i], 1);
      mbar_init(&sm.tail_done[i], 2);                            // both CTAs' tail warps
      mbar_init(&empty_bar[i], 1);
      sm.loads[i] = sm.tails[i] = 0;
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
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                                  // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem_base = sm.tmem_base;
  const int total = a.prob[0].tiles + (a.n_prob > 1 ? a.prob[1].tiles : 0);

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < total && ok && !*abort_flag; t += stride) {
        const WgradTile w = wgrad_tile(a, off, t);
        const WgradProblem& pr = a.prob[w.p];
        const int m = w.m + 128 * rank;
        const int nb = w.n / 64 + (pr.N - w.n > 128 ? 2 : 1) * rank;    // this CTA's half of B's features
        for (int k = 0; k < w.kn; k += KB) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, a.status, a.wait_ns)) { ok = false; break; }
          const bool tail = w.kn - k <= KB && (w.kn & 15);         // rows to zero
          uint32_t bar;
          if (tail) {
            mbar_arrive_expect_tx(&sm.tail_full[stage], C::STAGE_BYTES);
            bar = mapa_shared(smem_u32(&sm.tail_full[stage]), rank);
            ++sm.tails[stage];
          } else {
            if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * C::STAGE_BYTES);
            bar = mapa_shared(smem_u32(&full_bar[stage]), 0);
            ++sm.loads[stage];
          }
          if (pr.a_flat) {                                         // rows not a whole number of boxes wide
            tma_load_2d_pair(sA(stage), &pr.tmA, bar, m, w.k0 + k, pol);
            tma_load_2d_pair(sA(stage) + kChunkBytes, &pr.tmA, bar, m + 64, w.k0 + k, pol);
          } else {
            tma_load_3d_pair(sA(stage), &pr.tmA, bar, w.k0 + k, m / 64, pol);
          }
          tma_load_3d_pair(sB(stage), &pr.tmB, bar, w.k0 + k, nb, pol);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (*abort_flag)                                             // this CTA's tail loads; the others: below
        for (int i = 0; i < STAGES; ++i)
          if (sm.tails[i]) mbar_wait_drain(&sm.tail_full[i], (sm.tails[i] - 1) & 1u);
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      // Nothing but the wait stands between one block's MMAs and the next's:
      // their issue keeps only a few queued, and 700 cycles of bookkeeping a
      // block (512 of MMAs) cost a third of the rate.
      const uint64_t ad0 = mn_desc(smem_u32(sm.stage[0]));         // descriptor of stage 0's A
      int st = 0;
      uint32_t it = 0, full_par = 0, tail_par = 0;                 // parity of each stage's next wait, by barrier
      bool ok = true;
      for (int t = first; t < total && ok; t += stride, ++it) {
        const WgradTile w = wgrad_tile(a, off, t);
        const uint32_t idesc = make_idesc(1u, 256u, a.prob[w.p].N - w.n > 128 ? 256u : 128u) | kIdescAMn | kIdescBMn;
        const uint32_t d0 = tmem_base + (it & 1u) * 256;
        const int even = w.kn / KB, rest = w.kn - even * KB;       // blocks of 64 rows, and the last one's rows
        ok = mbar_wait(&tmem_empty[it & 1u], ((it >> 1) & 1u) ^ 1u, abort_flag, a.status, a.wait_ns);
        if (!ok) break;
        tc_fence_after();
        uint32_t acc = 0;
        for (int kb = 0; kb < even; ++kb) {
          ok = mbar_wait(&full_bar[st], (full_par >> st) & 1u, abort_flag, a.status, a.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = ad0 + st * (C::STAGE_BYTES >> 4), bd = ad + (C::PAIR >> 4);
#pragma unroll
          for (int kk = 0; kk < KB / 16; ++kk) {                   // 2048 B a step, in the descriptors' 16-byte units
            umma_bf16_pair(d0, ad + kk * 128, bd + kk * 128, idesc, acc);
            acc = 1;
          }
          umma_commit_pair(&empty_bar[st]);
          full_par ^= 1u << st;
          if (++st == STAGES) st = 0;
        }
        if (ok && rest > 0) {
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
          umma_commit_pair(&empty_bar[st]);
          if (++st == STAGES) st = 0;
        }
        if (ok) umma_commit_pair(&tmem_full[it & 1u]);
      }
      // all issued MMAs must finish before TMEM is released
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                       smem_u32(&sm.drain_bar))
                   : "memory");
      mbar_wait_drain(&sm.drain_bar, 0);
    }
  } else if (warp == 2 + EPIW) {
    // rows behind the segment's end in the last block: zeroed as soon as they land
    int stage = 0;
    uint32_t par = 0;
    for (int t = first; t < total; t += stride) {
      const WgradTile w = wgrad_tile(a, off, t);
      const int blocks = (max(w.kn, 0) + KB - 1) / KB;
      if (w.kn & 15) {
        const int st = (stage + blocks - 1) % STAGES;
        const int valid = w.kn - (blocks - 1) * KB;
        bool ok = true;
        if (lane == 0) ok = mbar_wait(&sm.tail_full[st], (par >> st) & 1u, abort_flag, a.status, a.wait_ns);
        if (__shfl_sync(0xffffffffu, ok ? 1 : 0, 0) == 0) break;
        par ^= 1u << st;
        const int nz = ((valid + 15) / 16 * 16 - valid) * 128;     // bytes per box: A's two boxes, then B's
        uint8_t* base = sA(st) + valid * 128;
        for (int i = lane * 16; i < nz; i += 512)
#pragma unroll
          for (int b = 0; b < 4; ++b) *reinterpret_cast<uint4*>(base + b * kChunkBytes + i) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive_first(&sm.tail_done[st]);
      }
      stage = (stage + blocks) % STAGES;
    }
  } else {
    const int q = warp & 3, half = (warp - 2) / 4;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    uint8_t* box = sm.out[warp - 2];
    const int cols = a.f32 ? 32 : 64;                              // columns of a 128-byte box row
    uint32_t it = 0;
    for (int t = first; t < total; t += stride, ++it) {
      const WgradTile w = wgrad_tile(a, off, t);
      const WgradProblem& pr = a.prob[w.p];
      const int width = pr.N - w.n > 128 ? 256 : 128;
      const int m = w.m + 128 * rank + 32 * q;                     // this warp's 32 features of A
      const uint32_t acc = lane_addr + (it & 1u) * 256;
      if (!mbar_wait(&tmem_full[it & 1u], (it >> 1) & 1u, abort_flag, a.status, a.wait_ns)) break;
      tc_fence_after();
      const bool empty = w.kn <= 0;
      // adding nothing needs no store, and rows past the matrix have none
      if (!(empty && a.accumulate) && m < pr.M) {
        for (int c = half * cols; c < width; c += 2 * cols) {
          float v[32], v2[32];
          if (!empty) {
            tmem_ld32(acc + c, v);
            if (!a.f32) tmem_ld32(acc + c + 32, v2);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = v2[j] = 0.0f;
          }
          // the last store of this box has been read
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
          uint8_t* row = box + lane * 128;
          if (a.f32) {
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
            const int y = w.g * pr.M + m;
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
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_first_relaxed(&tmem_empty[it & 1u]);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                                                  // neither CTA issues anything any more
  // After an abort one CTA may have loaded into a stage what the other had not
  // got to: complete the phases both started, arm the one only the second
  // started, so that every load has landed before either CTA leaves.
  if (rank == 0 && threadIdx.x == 0 && (*abort_flag || ld_cluster(&sm.abort_flag, 1) != 0)) {
    for (int i = 0; i < STAGES; ++i) {
      const uint32_t mine = sm.loads[i], theirs = ld_cluster(&sm.loads[i], 1);
      if (mine > theirs)
        asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&full_bar[i])),
                     "r"(C::STAGE_BYTES)
                     : "memory");
      else if (theirs > mine)
        mbar_arrive_expect_tx(&full_bar[i], C::STAGE_BYTES);
      const uint32_t n = mine > theirs ? mine : theirs;
      if (n) mbar_wait_drain(&full_bar[i], (n - 1) & 1u);
    }
  }
  cluster_sync();                                                  // nothing of either CTA is used any more
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// ========================================================================
// Router: d_logits from the gradients of the routing weights
// ========================================================================
// w_j = scale * s_j (/ sum_i s_i if normalised), s the softmax or sigmoid
// scores of the k chosen experts (the selection itself has no gradient):
//   ds_j = scale * dw_j, normalised: scale / S * (dw_j - sum_i dw_i s_i / S)
//   sigmoid: d_logit_e = s_e (1 - s_e) ds_e;  softmax: p_e (ds_e - sum_i p_i ds_i)
// with ds_e = 0 for experts not chosen. One warp per token: lane j holds slot
// j, lane l the experts l, l + 32, ... . Bound by its E logits' bytes.
__global__ void __launch_bounds__(256)
route_backward_kernel(int T, int E, int k, int scoring, int norm, float scale, const float* __restrict__ logits,
                      const int32_t* __restrict__ ids, const float* __restrict__ d_w,
                      const int32_t* __restrict__ slot_to_row, float* __restrict__ d_logits,
                      __nv_bfloat16* __restrict__ d_logits16, int32_t* status) {
  constexpr int PER = 8;                                           // E <= 256
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
  float p[PER];                                                    // softmax: this lane's probabilities
  float top = 0.0f, inv = 0.0f;
  if (scoring == MOE_SOFTMAX) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      p[i] = e < E ? lg[e] : -INFINITY;
      top = fmaxf(top, p[i]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      p[i] = expf(p[i] - top);
      sum += p[i];
    }
    inv = 1.0f / all_sum(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] *= inv;
  }
  // scores of the chosen experts, and the gradient of each
  const float s = id < 0 ? 0.0f : scoring == MOE_SOFTMAX ? expf(l_id - top) * inv : 1.0f / (1.0f + expf(-l_id));
  float ds = id < 0 ? 0.0f : scale * dw;
  if (norm) {
    const float S = all_sum(s);
    const float mean = all_sum(id < 0 ? 0.0f : dw * s) / S;
    ds = id < 0 ? 0.0f : scale / S * (dw - mean);
  }
  if (scoring == MOE_SIGMOID) ds *= s * (1.0f / (1.0f + expf(l_id)));   // s (1 - s), both without cancellation
  const float dot = scoring == MOE_SOFTMAX ? all_sum(ds * s) : 0.0f;
  float out[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) out[i] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int idj = __shfl_sync(0xffffffffu, id, j);
    const float dsj = __shfl_sync(0xffffffffu, ds, j);
#pragma unroll
    for (int i = 0; i < PER; ++i) out[i] += idj == lane + 32 * i ? dsj : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    if (e < E) {
      const float d = scoring == MOE_SOFTMAX ? p[i] * (out[i] - dot) : out[i];
      d_logits[static_cast<size_t>(t) * E + e] = d;
      if (d_logits16) d_logits16[static_cast<size_t>(t) * E + e] = __float2bfloat16_rn(d);
    }
  }
}

// ------------------------------------------------------------------------
// host-side launch helpers (called from api.cu)
// ------------------------------------------------------------------------
cudaError_t launch_train_gemm(int mode, const CUtensorMap& tmA, const TokenMaps& tmB, const TrainGemmArgs& a, int grid,
                              cudaStream_t stream) {
  const size_t smem = 3 * (4 * kChunkBytes + 256 * 128) + 1024;
  constexpr int W = 8;
  auto kern = mode == TRAIN_FORWARD ? train_gemm_kernel<TRAIN_FORWARD, W>
              : mode == TRAIN_HIDDEN ? train_gemm_kernel<TRAIN_HIDDEN, W> : train_gemm_kernel<TRAIN_ROWS, W>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  kern<<<grid, 64 + 32 * W, smem, stream>>>(tmA, tmB, a);
  return cudaGetLastError();
}

cudaError_t launch_row_w_grad(int rows, int n, const float* partial, const int32_t* offsets, int groups, float* d_row_w,
                              cudaStream_t stream) {
  row_w_grad_kernel<<<(rows + 255) / 256, 256, 0, stream>>>(rows, n, partial, offsets, groups, d_row_w);
  return cudaGetLastError();
}

cudaError_t launch_route_backward(int T, int E, int k, int scoring, int norm, float scale, const float* logits,
                                  const int32_t* ids, const float* d_w, const int32_t* slot_to_row, float* d_logits,
                                  void* d_logits16, int32_t* status, cudaStream_t stream) {
  route_backward_kernel<<<(T + 7) / 8, 256, 0, stream>>>(T, E, k, scoring, norm, scale, logits, ids, d_w, slot_to_row,
                                                         d_logits, reinterpret_cast<__nv_bfloat16*>(d_logits16), status);
  return cudaGetLastError();
}

cudaError_t launch_wgrad(const WgradArgs& a, int num_sms, cudaStream_t stream) {
  constexpr size_t smem = sizeof(WgradSmem);
  static_assert(smem <= 232448, "wgrad_kernel's shared memory exceeds an SM's");
  cudaError_t e = cudaFuncSetAttribute(wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int tiles = a.prob[0].tiles + (a.n_prob > 1 ? a.prob[1].tiles : 0);
  const int pairs = num_sms / 2 < tiles ? num_sms / 2 : tiles;
  wgrad_kernel<<<2 * pairs, WgradCfg::THREADS, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
