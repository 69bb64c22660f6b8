// Microscaled 4-bit floating point (MXFP4): E2M1 values (0, 0.5, 1, 1.5, 2, 3,
// 4, 6 and their negatives, two a byte, the first in the low half) with one
// E8M0 scale 2^(s - 127) per 32 consecutive values.
//
// Quantising a block: s - 127 = floor(log2 amax) - 2, clamped to [-127, 125]
// (2 is the exponent of the largest code, 6 = 1.5 * 2^2), s = 127 for a block
// of zeros; code = nearest of v / scale, ties to the even code, above 6 to 6.
// The division is by a power of two and so exact: codes depend on nothing but
// this definition. A block holding NaN or infinity gets s = 255 (NaN), which
// makes every product with it NaN.
//
// The product runs on the tensor cores' block-scaled form
// (tcgen05.mma kind::mxf4, K = 64 and two scales per row and instruction): the
// scales are applied inside the MMA, sums are fp32 in TMEM.
#include "mxfp4.cuh"

#include "segments.cuh"

namespace moe {

// ---------------------------------------------------------------- values
__device__ __forceinline__ uint32_t mx_scale_of(float amax) {
  const int field = static_cast<int>(__float_as_uint(amax) >> 23);   // amax >= 0; NaN and infinity: 255
  if (field == 255) return 255u;
  if (amax == 0.0f) return 127u;
  const int e = field - 127 - 2;                                     // subnormal: below the clamp as well
  return static_cast<uint32_t>(max(e, -127) + 127);
}
// 1 / scale as a float: exact (a NaN scale's blocks quantise against 1)
__device__ __forceinline__ float mx_inv_scale(uint32_t s) {
  return s == 255u ? 1.0f : __uint_as_float((254u - s) << 23);       // s <= 252
}
// eight values -> eight codes, value i in bits 4i..4i+3
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], float inv) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0] * inv), "f"(v[1] * inv), "f"(v[2] * inv), "f"(v[3] * inv), "f"(v[4] * inv), "f"(v[5] * inv),
        "f"(v[6] * inv), "f"(v[7] * inv));
  return r;
}
// |v|, with NaN as infinity, so that a maximum over a block keeps either
__device__ __forceinline__ float mx_mag(float v) { return v != v ? INFINITY : fabsf(v); }

// Four lanes hold a block of 32 values, eight each: its scale byte and this
// lane's codes. The largest magnitude and the scaling run on pairs of bf16 (the
// maximum keeps NaN; a power of two scales exactly, and what falls below bf16's
// smallest number is far below half a code).
__device__ __forceinline__ uint32_t mx_block(const uint4& u, uint32_t& scale) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  auto pair = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
  __nv_bfloat162 m2 = __hmax2_nan(__hmax2_nan(__habs2(pair(w[0])), __habs2(pair(w[1]))),
                                  __hmax2_nan(__habs2(pair(w[2])), __habs2(pair(w[3]))));
  uint32_t m = *reinterpret_cast<const uint32_t*>(&m2);
#pragma unroll
  for (int d = 1; d <= 2; d <<= 1) {
    m2 = __hmax2_nan(pair(m), pair(__shfl_xor_sync(0xffffffffu, m, d)));
    m = *reinterpret_cast<const uint32_t*>(&m2);
  }
  const float amax = __bfloat162float(__hmax_nan(__low2bfloat16(m2), __high2bfloat16(m2)));
  scale = mx_scale_of(amax);
  const __nv_bfloat162 inv = __float2bfloat162_rn(mx_inv_scale(scale));
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __hmul2(pair(w[i]), inv);
    const uint32_t x = *reinterpret_cast<const uint32_t*>(&p);
    f[2 * i] = __uint_as_float(x << 16);
    f[2 * i + 1] = __uint_as_float(x & 0xffff0000u);
  }
  return mx_codes8(f, 1.0f);
}

// ---------------------------------------------------------------- rows
// One warp per row and 1024 values, all four of its loads (16 bytes a lane) in
// flight at once, the CTA's eight warps on neighbouring rows, whose scale words
// [K / 128][rows] share sectors. Bound by HBM: 2 bytes read and 0.53 written per
// value, or the reverse. 4096 x 7168 (74 MB): 15 us, and 18 back; a warp per
// whole row took 20. Four or sixteen rows a CTA, 512 or 1792 values a warp:
// within 4 %.
constexpr int kMxRows = 8;                                           // rows (warps) per CTA
constexpr int kMxSteps = 4;                                          // of 256 values per warp
__global__ void __launch_bounds__(32 * kMxRows)
mx_quant_rows_kernel(int rows, int K, const uint4* a, int a_rows, const int32_t* src,
                     uint32_t* q, uint32_t* scale, int32_t* status) {
  launch_dependents_if_small();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kMxRows + (threadIdx.x >> 5);
  if (r >= rows) return;                                             // warp-uniform
  int from = src ? src[r] : r;
  const bool bad = from < 0 || from >= a_rows;
  if (bad) {                                                         // such a row becomes zeros
    if (lane == 0) flag_status(status, MOE_DEVSTAT_BAD_EXPERT_ID);
    from = 0;
  }
  const uint4* row = a + static_cast<size_t>(from) * (K / 8);
  uint32_t* qr = q + static_cast<size_t>(r) * (K / 8);
  const int c0 = blockIdx.y * (32 * kMxSteps) + lane;
  uint4 u[kMxSteps];
#pragma unroll
  for (int i = 0; i < kMxSteps; ++i) {
    const int c = c0 + 32 * i;
    u[i] = c < K / 8 && !bad ? row[c] : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kMxSteps; ++i) {
    const int c = c0 + 32 * i;
    uint32_t s;
    const uint32_t codes = mx_block(u[i], s);
    // the four blocks of 128 values: lanes 0, 4, 8, 12 and 16, 20, 24, 28
    uint32_t w = s << (8 * ((lane >> 2) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    if (c < K / 8) {
      qr[c] = codes;
      if ((lane & 15) == 0) scale[static_cast<size_t>(c / 16) * rows + r] = w;
    }
  }
}

// Two values' bits in bf16 (exact: two significant bits, and 2^-128 .. 1.5 *
// 2^127 are bf16 numbers).
__device__ __forceinline__ uint32_t mx_bf16x2(uint32_t codes, float sc) {
  // E2M1 magnitude m: 0, 0.5, 1, 1.5, 2, 3, 4, 6
  auto value = [&](uint32_t c) {
    const uint32_t m = c & 7u;
    const float x = m < 2 ? 0.5f * static_cast<float>(m) : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
    return (c & 8u) ? -x * sc : x * sc;
  };
  const __nv_bfloat162 h = __floats2bfloat162_rn(value(codes & 15u), value((codes >> 4) & 15u));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__global__ void __launch_bounds__(32 * kMxRows)
mx_dequant_rows_kernel(int rows, int K, const uint32_t* q, const uint32_t* scale,
                       uint4* out) {
  launch_dependents_if_small();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kMxRows + (threadIdx.x >> 5);
  if (r >= rows) return;
  const uint32_t* qr = q + static_cast<size_t>(r) * (K / 8);
  uint4* o = out + static_cast<size_t>(r) * (K / 8);
  const int c0 = blockIdx.y * (32 * kMxSteps) + lane;
  uint32_t code[kMxSteps], w[kMxSteps];
#pragma unroll
  for (int i = 0; i < kMxSteps; ++i) {
    const int c = c0 + 32 * i;
    code[i] = c < K / 8 ? qr[c] : 0u;
    w[i] = c < K / 8 ? scale[static_cast<size_t>(c / 16) * rows + r] : 0u;
  }
#pragma unroll
  for (int i = 0; i < kMxSteps; ++i) {
    const int c = c0 + 32 * i;
    const uint32_t s = (w[i] >> (8 * ((lane >> 2) & 3))) & 255u;
    // 2^(s - 127): s = 0 is the subnormal 2^-127, s = 255 NaN
    const float sc = s == 255u ? __uint_as_float(0x7fc00000u) : s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
    uint4 v;
    v.x = mx_bf16x2(code[i], sc);
    v.y = mx_bf16x2(code[i] >> 8, sc);
    v.z = mx_bf16x2(code[i] >> 16, sc);
    v.w = mx_bf16x2(code[i] >> 24, sc);
    if (c < K / 8) o[c] = v;
  }
}

// Weights (once, when a layer is built): one warp per row; scales in the order
// the GEMM copies into shared memory, per 128 rows x 128 columns row r's word
// at (r % 32) * 16 + (r / 32) * 4.
__global__ void __launch_bounds__(256)
mx_quant_weights_kernel(long long n_rows, int N, int K, const uint4* __restrict__ w, uint32_t* __restrict__ q,
                        uint8_t* __restrict__ scale) {
  const int lane = threadIdx.x & 31;
  const long long gr = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (gr >= n_rows) return;
  const int rr = static_cast<int>(gr % 128);
  uint32_t* sc = reinterpret_cast<uint32_t*>(scale + (gr / 128) * static_cast<size_t>(K / 128) * 512 + (rr % 32) * 16 +
                                             (rr / 32) * 4);
  for (int c0 = 0; c0 < K / 8; c0 += 32) {
    const int c = c0 + lane;
    uint32_t s;
    const uint32_t codes = mx_block(c < K / 8 ? w[gr * (K / 8) + c] : make_uint4(0u, 0u, 0u, 0u), s);
    uint32_t word = s << (8 * ((lane >> 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (c < K / 8) {
      q[gr * (K / 8) + c] = codes;
      if ((lane & 15) == 0) sc[static_cast<size_t>(c / 16) * 128] = word;
    }
  }
}

// ---------------------------------------------------------------- product
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::mxf4: E2M1 x E2M1 (1 at bits 7 and 10), N / 8 at
// 17, UE8M0 scales (bit 23), M / 128 at 27; the scale pair used (bytes 0-1 or
// 2-3 of a row's word) at bits 4 (B) and 29 (A).
__device__ __forceinline__ uint32_t mxf4_idesc(uint32_t M, uint32_t N, uint32_t pair) {
  return (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (1u << 23) | ((M >> 7) << 27) | ((2 * pair) << 4) | ((2 * pair) << 29);
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z, int32_t t, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(t), "l"(policy)
      : "memory");
}

constexpr int kMxEpi = 8;                                            // epilogue warps
constexpr int kMxThreads = 32 * (8 + kMxEpi);
constexpr int kMxMaxStages = 4;
constexpr uint32_t kMxA = 256 * 128;                                 // 256 weight rows x 256 values
constexpr uint32_t kMxSfa = 2048;                                    // their scales
__host__ __device__ constexpr uint32_t mx_stage_bytes(int bn) { return kMxA + kMxSfa + static_cast<uint32_t>(bn) * 128u; }
// Dynamic shared memory of a launch, and of the largest one mx_tile gives.
constexpr size_t mx_smem(int bn, int stages) { return static_cast<size_t>(stages) * mx_stage_bytes(bn) + 1024; }
constexpr size_t kMxSmemMax = mx_smem(192, mx_stages(192));
static_assert(mx_smem(32, mx_stages(32)) <= kMxSmemMax && mx_smem(64, mx_stages(64)) <= kMxSmemMax,
              "192 rows a tile take the most shared memory");

// Tiles as in the forward GEMMs: 256 weight rows (gate and up rows of 128
// features, or 256 rows of w2) as the MMA's A, up to bn_max rows of a segment
// as B, accumulated side by side in TMEM columns [0, bn) and [bn, 2 bn). A
// stage is 256 values of K: the weights' codes, their scales and the rows' codes
// by TMA, one box each, into shared memory, the rows' scales from L2. Four warps, one for each
// quarter of the TMEM lanes, then write all scales to 32 TMEM columns of the
// stage's own (2 bn + 32 * stage ..): lane l of column c has the word (four
// scales, 128 values) of row 32 c + l, the same in all four quarters. (Copied
// from shared memory by tcgen05.cp, which the MMAs wait for in line, 8 rows on
// each of 64 V3 experts took 268 us.)
//   warp 0 TMA, warp 1 TMEM and MMAs, warps 4..7 the scales, warps 8..15 the
//   epilogue: gate/up quantises h = SiLU(g) u, a warp's 32 features being one
//   block of 32, through a shared tile so that a lane has one row's block.
// The down epilogue reads its accumulators into registers, hands them back and
// stores while the next tile's products run (107 us otherwise, 97 with it, for the
// second case below).
// Measured on B200 at V3 widths, gate/up and down: 8 rows on each of 64 experts
// 152 and 79 us, bound by the weights' bytes (4.25 bits a value; 6.6 and 6.3 TB/s);
// 256 rows on each of 32 162 and 97 us (3.0 and 2.5 PFLOP/s), where with the
// epilogue left out 148 and 73 remain and half the MMAs change little: 1.4 GB of
// operands come from L2 in gate/up, near 10 TB/s.
template <bool GATE_UP>
__global__ void __launch_bounds__(kMxThreads, 1)
mx_gemm_kernel(const __grid_constant__ MxMaps maps, const MxGemmArgs a) {
  extern __shared__ __align__(1024) uint8_t dsmem[];
  __shared__ SegSched sched;
  __shared__ __align__(16) float tile_s[kMxEpi][32 * 33];
  __shared__ uint64_t full_bar[kMxMaxStages], sfa_bar[kMxMaxStages], scaled_bar[kMxMaxStages], empty_bar[kMxMaxStages];
  __shared__ uint64_t tmem_full, tmem_empty, drain_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int issued_parity[kMxMaxStages];
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  const uint32_t bn = static_cast<uint32_t>(a.bn_max);
  const uint32_t stage_bytes = mx_stage_bytes(a.bn_max);
  const int stages = a.stages;
  auto sA = [&](int st) { return smem + st * stage_bytes; };
  auto sB = [&](int st) { return smem + st * stage_bytes + kMxA; };
  auto sSfa = [&](int st) { return smem + st * stage_bytes + kMxA + bn * 128u; };
  const SegProblem sp{a.rows, a.groups, a.offsets, a.n_mblk, a.bn_max, 16, a.status};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMxMaxStages; ++i) {
      mbar_init(&full_bar[i], 1);                                    // the codes have landed
      mbar_init(&sfa_bar[i], 1);                                     // the weights' scales have
      mbar_init(&scaled_bar[i], 4);                                  // the scale warps have written TMEM
      mbar_init(&empty_bar[i], 1);
      issued_parity[i] = -1;
    }
    mbar_init(&tmem_full, 1);
    mbar_init(&tmem_empty, kMxEpi);                                  // one arrival per epilogue warp
    mbar_init(&drain_bar, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.w_scale);
    for (int i = 0; i < a.bn_max / 16; ++i) tma_prefetch_desc(&maps.rows[i]);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_s, 512);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  griddep_wait();
  if (warp == 3) build_schedule(sched, sp, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_s;
  const int total = total_tiles(sched, sp);
  const int k128 = a.K / 128;                                        // blocks of 128 values
  const int nk = (k128 + 1) / 2;                                     // stages per tile

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_once = policy_evict_first();
      const uint64_t pol_reuse = policy_evict_normal();
      const uint64_t pol_x = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      int g = 0;
      for (int t = blockIdx.x; t < total && !abort_flag; t += gridDim.x) {
        const SegTile ti = decode_tile(sched, sp, t, g);
        // the tile's weight rows: GATE_UP [2 groups][I], else [groups * H / 128][128]
        const int y = GATE_UP ? ti.mb * 128 : 0, z = GATE_UP ? 2 * ti.g : 2 * (ti.g * a.n_mblk + ti.mb);
        const CUtensorMap* mB = &maps.rows[ti.N / 16 - 1];
        const uint64_t pol_w = ti.ntb > 1 ? pol_reuse : pol_once;
        bool ok = true;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_flag, a.status, a.wait_ns)) { ok = false; break; }
          uint64_t* fb = &full_bar[stage];
          mbar_arrive_expect_tx(&sfa_bar[stage], kMxSfa);
          tma_load_4d(sSfa(stage), &maps.w_scale, &sfa_bar[stage], 0, 2 * kb, GATE_UP ? ti.mb : z, GATE_UP ? z : 0, pol_w);
          mbar_arrive_expect_tx(fb, kMxA + static_cast<uint32_t>(ti.N) * 128u);
          tma_load_3d(sA(stage), &maps.w, fb, kb * 128, y, z, pol_w);
          tma_load_2d(sB(stage), mB, fb, kb * 128, ti.row0, pol_x);
          issued_parity[stage] = static_cast<int>(phase);
          if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
      }
    }
  } else if (warp >= 4 && warp < 8) {
    const int q = warp & 3;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    int g = 0;
    for (int t = blockIdx.x; t < total && ok && !abort_flag; t += gridDim.x) {
      const SegTile ti = decode_tile(sched, sp, t, g);
      // columns [A0 kh0: 4][A0 kh1: 4][A1: 8][B kh0: 8][B kh1: 8]
      uint32_t x[16];                                                // the rows' words of the next block
      auto fetch = [&](int kb) {
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          const int kk = 2 * kb + kh;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int r = c * 32 + lane;                             // rows behind the tile's: scale 1, not used
            x[8 * kh + c] = kk < k128 && r < ti.n_valid
                                ? a.b_scale[static_cast<size_t>(kk) * a.rows + ti.row0 + r] : 0x7f7f7f7fu;
          }
        }
      };
      fetch(0);
      for (int kb = 0; kb < nk; ++kb) {
        ok = mbar_wait_warp(&sfa_bar[stage], phase, &abort_flag, a.status, a.wait_ns);
        if (!ok) break;
        uint32_t w[32];
        const uint4* sf = reinterpret_cast<const uint4*>(sSfa(stage)) + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) {                                // [A0 kh0][A0 kh1][A1 kh0][A1 kh1]
          const uint4 y = sf[32 * i];
          w[4 * i] = y.x; w[4 * i + 1] = y.y; w[4 * i + 2] = y.z; w[4 * i + 3] = y.w;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) w[16 + i] = x[i];
        tc_fence_after();
        tmem_st32(tmem_base + (static_cast<uint32_t>(32 * q) << 16) + 2 * bn + 32u * stage, w);
        if (kb + 1 < nk) fetch(kb + 1);                              // in flight while the store completes
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&scaled_bar[stage]);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, it = 0;
      const uint64_t ad0 = sw128_desc(smem_u32(sA(0))), bd0 = sw128_desc(smem_u32(sB(0)));
      int g = 0;
      for (int t = blockIdx.x; t < total && !abort_flag; t += gridDim.x, ++it) {
        const SegTile ti = decode_tile(sched, sp, t, g);
        const uint32_t id0 = mxf4_idesc(128u, static_cast<uint32_t>(ti.N), 0u);
        const uint32_t id1 = mxf4_idesc(128u, static_cast<uint32_t>(ti.N), 1u);
        if (!mbar_wait(&tmem_empty, (it & 1u) ^ 1u, &abort_flag, a.status, a.wait_ns)) break;
        tc_fence_after();
        bool ok = true;
        uint32_t acc = 0;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&full_bar[stage], phase, &abort_flag, a.status, a.wait_ns) ||
              !mbar_wait(&scaled_bar[stage], phase, &abort_flag, a.status, a.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sf = tmem_base + 2 * bn + 32u * stage;      // [A0: 8][A1: 8][B: 16] columns
          const uint64_t ad = ad0 + stage * (stage_bytes >> 4), bd = bd0 + stage * (stage_bytes >> 4);
          const int halves = min(2, k128 - 2 * kb);
          for (int kh = 0; kh < halves; ++kh) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {                            // 64 values: 32 B, 2 descriptor units
              const uint64_t k = static_cast<uint64_t>(2 * (2 * kh + p));
              const uint32_t id = p ? id1 : id0;
              umma_mxf4(tmem_base, ad + k, bd + k, id, sf + kh * 4, sf + 16 + kh * 8, acc);
              umma_mxf4(tmem_base + bn, ad + (128 * 128 >> 4) + k, bd + k, id, sf + 8 + kh * 4, sf + 16 + kh * 8, acc);
              acc = 1;
            }
          }
          umma_commit(&empty_bar[stage]);
          if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        umma_commit(&tmem_full);
      }
      umma_commit(&drain_bar);   // all issued MMAs must finish before TMEM is released
      mbar_wait_drain(&drain_bar, 0);
    }
  } else if (warp >= 8) {
    const int q = warp & 3;
    const int half = (warp - 8) / 4;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    float* ts = tile_s[warp - 8];
    uint32_t it = 0;
    int g = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x, ++it) {
      const SegTile ti = decode_tile(sched, sp, t, g);
      const int nchunk = (ti.N + 31) / 32;
      float* ws = ts + 512;                                          // down: the rows' weights, behind the store tile
      if (!GATE_UP) {
        for (int r = lane; r < 32 * nchunk; r += 32)
          ws[r] = r < ti.n_valid ? (a.row_w ? a.row_w[ti.row0 + r] : 1.0f) : 0.0f;
        __syncwarp();
      }
      if (!mbar_wait_warp(&tmem_full, it & 1u, &abort_flag, a.status, a.wait_ns)) break;
      tc_fence_after();
      auto done_reading = [&] {                                      // the next tile's MMAs may start
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tmem_empty);
      };
      if (GATE_UP) {
        if (half >= nchunk) done_reading();
        uint8_t* out = reinterpret_cast<uint8_t*>(a.out);
        for (int c = half; c < nchunk; c += 2) {
          float g[32], u[32];
          tmem_ld32(lane_addr + c * 32, g);
          tmem_ld32(lane_addr + bn + c * 32, u);
          tmem_ld_wait();
          if (c + 2 >= nchunk) done_reading();
#pragma unroll
          for (int j = 0; j < 32; ++j) ts[j * 33 + lane] = silu(g[j]) * u[j];
          __syncwarp();
          // lane = row: its 32 features of this warp are one block
          float m = 0.0f;
#pragma unroll
          for (int f = 0; f < 32; ++f) {
            g[f] = ts[lane * 33 + f];
            m = fmaxf(m, mx_mag(g[f]));
          }
          const uint32_t s = mx_scale_of(m);
          const float inv = mx_inv_scale(s);
          uint32_t code[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = g[8 * i + e];
            code[i] = mx_codes8(v, inv);
          }
          const int r = c * 32 + lane;
          if (r < ti.n_valid) {
            const size_t row = static_cast<size_t>(ti.row0 + r);
            *reinterpret_cast<uint4*>(out + row * (a.out_ld / 2) + ti.mb * 64 + q * 16) =
                make_uint4(code[0], code[1], code[2], code[3]);
            a.out_scale[(static_cast<size_t>(ti.mb) * a.rows + row) * 4 + q] = static_cast<uint8_t>(s);
          }
          __syncwarp();
        }
      } else {
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out);
        __nv_bfloat16* stg = reinterpret_cast<__nv_bfloat16*>(ts);
        // this warp: 32 features of sub-tile `half`, all chunks of rows; read (four
        // chunks held at once), then stored while the next tile's products run
        const uint32_t acc = lane_addr + half * bn;
        const int feat0 = ti.mb * 256 + half * 128 + 32 * q;
        uint32_t p[4][16];
        auto read = [&](int c, uint32_t (&to)[16]) {
          float v[32];
          tmem_ld_frag(acc + c * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 w = *reinterpret_cast<const float2*>(ws + c * 32 + frag_row(lane, (k >> 1) & 3, 0));
            to[k] = pack_bf16(v[2 * k] * w.x, v[2 * k + 1] * w.y);
          }
        };
        auto put = [&](int c, const uint32_t (&from)[16]) {
          store_frag(stg, from, lane, out, static_cast<size_t>(a.out_ld), ti.row0 + c * 32, ti.n_valid - c * 32, feat0);
        };
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < nchunk) read(c, p[c]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (c + 4 < nchunk) {
            put(c, p[c]);
            read(c + 4, p[c]);
          }
        done_reading();
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < nchunk) put(c + 4 < nchunk ? c + 4 : c, p[c]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (abort_flag && warp == 0 && lane == 0) {                        // every copy issued lands before the CTA leaves
    for (int i = 0; i < kMxMaxStages; ++i) {
      if (issued_parity[i] < 0) continue;
      mbar_wait_drain(&sfa_bar[i], static_cast<uint32_t>(issued_parity[i]));
      mbar_wait_drain(&full_bar[i], static_cast<uint32_t>(issued_parity[i]));
    }
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem_base, 512);
}

// ---------------------------------------------------------------- launches
cudaError_t launch_mx_gemm(bool gate_up, const MxMaps& maps, const MxGemmArgs& a, int grid, cudaStream_t stream) {
  auto kern = gate_up ? mx_gemm_kernel<true> : mx_gemm_kernel<false>;
  // The limit belongs to the kernel, not to the launch: it is always the largest, so
  // that another host thread's smaller call cannot lower it before this launch.
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMxSmemMax));
  if (e != cudaSuccess) return e;
  return launch_after(kern, grid, kMxThreads, mx_smem(a.bn_max, a.stages), stream, maps, a);
}

static dim3 mx_rows_grid(int rows, int K) {
  return dim3(static_cast<unsigned>((rows + kMxRows - 1) / kMxRows),
              static_cast<unsigned>((K + 256 * kMxSteps - 1) / (256 * kMxSteps)));
}
cudaError_t launch_mx_quant_rows(int rows, int K, const void* a, int a_rows, const int32_t* src, void* q, void* scale,
                                 int32_t* status, cudaStream_t stream) {
  return launch_after(mx_quant_rows_kernel, mx_rows_grid(rows, K), 32 * kMxRows, 0, stream, rows, K,
                      static_cast<const uint4*>(a), a_rows, src, static_cast<uint32_t*>(q), static_cast<uint32_t*>(scale),
                      status);
}
cudaError_t launch_mx_dequant_rows(int rows, int K, const void* q, const void* scale, void* out, cudaStream_t stream) {
  return launch_after(mx_dequant_rows_kernel, mx_rows_grid(rows, K), 32 * kMxRows, 0, stream, rows, K,
                      static_cast<const uint32_t*>(q), static_cast<const uint32_t*>(scale), static_cast<uint4*>(out));
}
cudaError_t launch_mx_quant_weights(int batch, int N, int K, const void* w, void* q, void* scale, cudaStream_t stream) {
  const long long n = static_cast<long long>(batch) * N;
  mx_quant_weights_kernel<<<static_cast<unsigned>((n + 7) / 8), 256, 0, stream>>>(
      n, N, K, static_cast<const uint4*>(w), static_cast<uint32_t*>(q), static_cast<uint8_t*>(scale));
  return cudaGetLastError();
}

}  // namespace moe
