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
  int tb;               // this tile's token block in the segment
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
  ti.tb = tb;
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

// Token rows of one stage (a multiple of 16, at most 256) are fetched with at
// most one box of each size 256, 128, 64, 32, 16: the binary digits of
// rows / 16. Returns rows loaded.
template <typename LoadFn>
__device__ __forceinline__ int load_token_rows(int rows, LoadFn&& load) {
  int off = 0;
#pragma unroll
  for (int i = 0; i < kTokBoxes; ++i) {
    const int box = 256 >> i;
    if (rows - off >= box) { load(i, off); off += box; }
  }
  return off;
}

// Writes NT tokens x 32 features (thread = feature lane, v[j] = token j) to
// out[(row0 + j) * ld + feat0 + lane] through a per-warp shared tile, so that
// every global store is a 16-byte vector (4 lanes cover one token's 32
// features). Tokens j >= n_rows are not written.
template <int NT>
__device__ __forceinline__ void store_tile(__nv_bfloat16* stage, const float (&v)[NT], int lane,
                                           __nv_bfloat16* out, size_t ld, int row0, int n_rows, int feat0) {
#pragma unroll
  for (int j = 0; j < NT; ++j) stage[j * 32 + lane] = __float2bfloat16_rn(v[j]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NT / 8; ++i) {
    const int t = (lane >> 2) + 8 * i;
    const int seg = lane & 3;
    if (t < n_rows) {
      const uint4 val = *reinterpret_cast<const uint4*>(stage + t * 32 + seg * 8);
      *reinterpret_cast<uint4*>(out + static_cast<size_t>(row0 + t) * ld + feat0 + seg * 8) = val;
    }
  }
  __syncwarp();
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
