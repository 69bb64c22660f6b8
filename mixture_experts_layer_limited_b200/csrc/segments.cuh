// Launches, tile loads and stores shared by the training and the 4-bit grouped GEMM
// kernels.
#pragma once

#include "schedule.cuh"
#include "train.cuh"

namespace moe {

// Launch with programmatic stream serialization: the kernel may start while the
// one before it in the stream still runs, so it sets up its barriers and TMEM
// beside that one's end and calls griddep_wait() before it touches global
// memory. The training and 4-bit calls are chains of such kernels, a few
// microseconds each where rows are few.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int block, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// For kernels of many small CTAs: lets the next kernel start early only where
// each SM has one CTA at most; beside more of them its CTAs would take the free
// places unevenly (4096 rows to 4 bits and back: 60 us instead of 48).
__device__ __forceinline__ void launch_dependents_if_small() {
  if (gridDim.x * gridDim.y <= 148) griddep_launch_dependents();
}

// ---- 32 features x 32 rows of an accumulator, as the tensor cores' fragments
// A warp's 32 TMEM lanes (features) x 32 columns (rows of the output): thread t
// holds, in v[16 h + 4 i + 2 s + e], feature 16 h + 8 s + t / 4 of row
// 8 i + 2 (t % 4) + e. Two rows (e) packed to bf16 are what stmatrix and ldmatrix
// take, which transpose 8 x 8 blocks on the way, so that the output's rows, whose
// features are contiguous, go through shared memory in 16-byte pieces (with one
// feature per thread they would go in 2-byte ones, eight times as many).
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr + (static_cast<uint32_t>(16 * h) << 16))
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[16 * h + i] = __uint_as_float(r[i]);
  }
}
// Stores 32 columns of this warp's 32 TMEM lanes, one lane a thread.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// The row of v[16 h + 4 i + 2 s + e] for thread t.
__device__ __forceinline__ int frag_row(int lane, int i, int e) { return 8 * i + 2 * (lane & 3) + e; }

// Packed fragments: p[8 h + 2 i + s] holds the rows e = 0 (low half) and 1.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void pack_frag(const float (&v)[32], uint32_t (&p)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) p[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
}
// Byte offset of 16-byte piece `seg` (8 features) of row r in the warp's 2 KB tile.
__device__ __forceinline__ uint32_t tile_piece(int r, int seg) {
  return static_cast<uint32_t>(r * 64 + ((seg ^ ((r >> 1) & 3)) << 4));
}
// Stores packed fragments as rows [row0, +n_rows) x 32 features from feat0.
__device__ __forceinline__ void store_frag(__nv_bfloat16* tile, const uint32_t (&p)[16], int lane, __nv_bfloat16* out,
                                           size_t ld, int row0, int n_rows, int feat0) {
  const uint32_t base = smem_u32(tile);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     base + tile_piece(8 * i + (lane & 7), lane >> 3)),
                 "r"(p[2 * i]), "r"(p[2 * i + 1]), "r"(p[8 + 2 * i]), "r"(p[8 + 2 * i + 1])
                 : "memory");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (lane >> 2) + 8 * i, seg = lane & 3;
    if (r < n_rows)
      *reinterpret_cast<uint4*>(out + static_cast<size_t>(row0 + r) * ld + feat0 + seg * 8) =
          *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(tile) + tile_piece(r, seg));
  }
  __syncwarp();
}

// 32 rows x 32 features of a bf16 matrix: fetched (rows >= n_rows as zeros) ..
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
// .. and turned into packed fragments through the warp's tile.
__device__ __forceinline__ void spread_frag(__nv_bfloat16* tile, const TileRegs& t, int lane, uint32_t (&p)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(tile) + tile_piece((lane >> 2) + 8 * i, lane & 3)) = t.r[i];
  __syncwarp();
  const uint32_t base = smem_u32(tile);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(p[2 * i]), "=r"(p[2 * i + 1]), "=r"(p[8 + 2 * i]), "=r"(p[8 + 2 * i + 1])
                 : "r"(base + tile_piece(8 * i + (lane & 7), lane >> 3))
                 : "memory");
  __syncwarp();
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t p) {
  return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}
// The eight rows' values of a per-row vector that thread t's fragments need:
// w[2 i + e], 0 for rows >= n_rows; nullptr: `none`.
__device__ __forceinline__ void frag_row_values(const float* src, int n_rows, int lane, float none, float (&w)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = frag_row(lane, k >> 1, k & 1);
    w[k] = r < n_rows ? (src ? src[r] : none) : 0.0f;
  }
}

// mbar_wait for a whole warp: one lane waits, so that all lanes go on, or give
// up after an abort, together.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status,
                                               uint64_t limit_ns) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_flag, status, limit_ns) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

}  // namespace moe
