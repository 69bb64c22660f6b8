// The tile schedule over expert segments and the tile loads and stores shared
// by the training and the 4-bit grouped GEMM kernels. Tiles are (expert g,
// feature block mb, row block tb), at most bn_max rows each, as in the forward
// GEMMs; a segment that does not lie in the rows is cut to them and flagged.
#pragma once

#include "train.cuh"

namespace moe {

constexpr int kMaxGroups = 512;

struct SegTile {
  int g, mb, row0, n_valid, N;
  int ntb;              // token blocks of this segment
};

// Token blocks per rasterisation chunk: inside a segment, tiles run in chunks
// of up to kTbChunk token blocks x all weight blocks, token block innermost,
// so CTAs running side by side share the weight block (HBM once, then L2)
// and the chunk's token blocks (L2).
constexpr int kTbChunk = 8;

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

// A grouped GEMM as the schedule sees it.
struct SegProblem {
  int32_t rows, groups;
  const int32_t* offsets;   // [groups + 1] or nullptr (one segment of all rows)
  int32_t n_mblk;           // feature blocks per group
  int32_t bn_max;           // max rows per tile (multiple of 32, <= 256)
  int32_t unit;             // tiles are computed in multiples of this many rows (16 or 32)
  int32_t* status;
};

// Per-CTA copy of the tile schedule: each group's first tile and first row.
struct SegSched {
  int tile_start[kMaxGroups + 1];
  int seg_start[kMaxGroups + 1];
};

__device__ __forceinline__ int tiles_of(int n, int bn_max, int n_mblk) {
  return n <= 0 ? 0 : ((n + bn_max - 1) / bn_max) * n_mblk;
}

// Warp-cooperative build of the schedule (called by one warp).
__device__ __forceinline__ void build_schedule(SegSched& s, const SegProblem& a, int lane) {
  int carry = 0;
  for (int base = 0; base < a.groups; base += 32) {
    const int g = base + lane;
    int st = 0, n = 0;
    if (g < a.groups) {
      if (a.offsets) {
        st = a.offsets[g];
        int end = a.offsets[g + 1];
        if (st < 0 || end < st || end > a.rows) {       // a segment outside the rows: flagged, cut to them
          flag_status(a.status, MOE_DEVSTAT_BAD_EXPERT_ID);
          st = min(max(st, 0), a.rows);
          end = min(max(end, st), a.rows);
        }
        n = end - st;
      } else {
        st = 0;
        n = a.rows;
      }
    }
    int t = (g < a.groups) ? tiles_of(n, a.bn_max, 1) : 0;   // token blocks
    int incl = t;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (g < a.groups) {
      s.tile_start[g] = (carry + incl - t) * a.n_mblk;
      s.seg_start[g] = st;
    }
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) {
    s.tile_start[a.groups] = carry * a.n_mblk;
    s.seg_start[a.groups] = a.offsets ? min(max(a.offsets[a.groups], 0), a.rows) : a.rows;
  }
}

// a / b for 0 <= a, 0 < b: a float quotient where it is exact (a < 2^20: its
// error is below a quarter). Every role of a CTA decodes every tile, the loads'
// and the MMAs' threads between two tiles' work: integer divisions there cost a
// thousand cycles a tile.
__device__ __forceinline__ int quick_div(int a, int b) {
  return a < (1 << 20) ? __float2int_rz(__fdividef(static_cast<float>(a) + 0.5f, static_cast<float>(b))) : a / b;
}

// Tile `local` of a segment of n rows starting at row seg0 (group g).
__device__ __forceinline__ SegTile decode_in_segment(const SegProblem& a, int g, int seg0, int n, int local) {
  SegTile ti;
  ti.g = g;
  const int ntb = quick_div(n + a.bn_max - 1, a.bn_max);
  const int bn = (quick_div(n + ntb - 1, ntb) + a.unit - 1) & ~(a.unit - 1);
  const int chunk_tiles = kTbChunk * a.n_mblk;
  const int chunk = ntb <= kTbChunk ? 0 : quick_div(local, chunk_tiles);
  const int r = local - chunk * chunk_tiles;
  const int c_tb = min(kTbChunk, ntb - chunk * kTbChunk);   // token blocks in this chunk
  ti.mb = quick_div(r, c_tb);
  const int tb = chunk * kTbChunk + (r - ti.mb * c_tb);
  ti.ntb = ntb;
  ti.row0 = seg0 + tb * bn;
  ti.n_valid = min(bn, n - tb * bn);
  ti.N = (ti.n_valid + a.unit - 1) & ~(a.unit - 1);
  return ti;
}

// Tile t; g: the group of the caller's last tile (0 at first; t only grows).
__device__ __forceinline__ SegTile decode_tile(const SegSched& s, const SegProblem& a, int t, int& g) {
  while (t >= s.tile_start[g + 1]) ++g;
  return decode_in_segment(a, g, s.seg_start[g], s.seg_start[g + 1] - s.seg_start[g], t - s.tile_start[g]);
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

// SiLU(g) = g * sigmoid(g). Fast division: for g < -88 the exponential
// overflows to inf and the quotient is the correct limit (-0).
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

}  // namespace moe
