// The tile schedule over expert segments, shared by every grouped GEMM (forward,
// training, 4-bit). Tiles are (expert g, feature block mb, row block tb), at most
// bn_max rows each.
#pragma once

#include "kernels.cuh"

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

// A grouped GEMM as the schedule sees it (GemmArgs has the same fields but for
// `unit`, see seg_unit).
struct SegProblem {
  int32_t rows, groups;
  const int32_t* offsets;   // [groups + 1] or nullptr (one segment of all rows)
  int32_t n_mblk;           // feature blocks per group
  int32_t bn_max;           // max rows per tile (multiple of 32, <= 256)
  int32_t unit;             // tiles are computed in multiples of this many rows (16 or 32)
  int32_t* status;
};
__device__ __forceinline__ int seg_unit(const SegProblem& a) { return a.unit; }
__device__ __forceinline__ int seg_unit(const GemmArgs&) { return 16; }

// Per-CTA copy of the tile schedule: each group's first token block (over all
// groups) and first row. A group's first tile is its first token block times the
// problem's feature blocks.
struct SegSched {
  int tb_start[kMaxGroups + 1];
  int seg_start[kMaxGroups + 1];
};

__device__ __forceinline__ int tiles_of(int n, int bn_max, int n_mblk) {
  return n <= 0 ? 0 : ((n + bn_max - 1) / bn_max) * n_mblk;
}

// Segments lie one after the other inside the rows, whatever the offsets say: a
// start outside the rows is cut to them, one that falls to the largest before it,
// and either is flagged. A kernel first takes the offsets as they are, looking at
// each segment for itself (seg_lies); only where one fails does a warp go through
// all of them (tiny layer 91.8 us; always cutting 93.4).
__device__ __forceinline__ bool seg_lies(int start, int end, int rows) { return 0 <= start && start <= end && end <= rows; }
__device__ __forceinline__ void cut_starts(int* start, const int32_t* offsets, int groups, int rows, int32_t* status, int lane) {
  int most = 0;                                          // the largest start so far
  for (int base = 0; base <= groups; base += 32) {
    const int g = base + lane;
    int st = g > groups ? 0 : min(max(offsets[g], 0), rows);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, st, d);
      if (lane >= d) st = max(st, v);
    }
    st = max(st, most);
    if (g <= groups) start[g] = st;
    most = __shfl_sync(0xffffffffu, st, 31);
  }
  if (lane == 0) flag_status(status, MOE_DEVSTAT_BAD_EXPERT_ID);
  __syncwarp();
}

// Each group's first token block and row from the segments' starts (nullptr: one
// segment of all rows); whether all of them lie in the rows. Called by one warp.
__device__ __forceinline__ bool fill_schedule(SegSched& s, const int* starts, int groups, int rows, int bn_max, int lane) {
  int carry = 0;
  bool lie = true;
  for (int base = 0; base < groups; base += 32) {
    const int g = base + lane;
    int st = 0, n = 0;
    if (g < groups) {
      if (starts) {
        st = starts[g];
        const int end = starts[g + 1];
        lie = lie && seg_lies(st, end, rows);
        n = end - st;
      } else {
        n = rows;
      }
    }
    const int t = tiles_of(n, bn_max, 1);                // token blocks
    int incl = t;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (g < groups) {
      s.tb_start[g] = carry + incl - t;
      s.seg_start[g] = st;
    }
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) {
    s.tb_start[groups] = carry;
    s.seg_start[groups] = starts ? starts[groups] : rows;
  }
  return __all_sync(0xffffffffu, lie);
}
static __device__ __noinline__ void cut_schedule(SegSched& s, const int32_t* offsets, int groups, int rows, int bn_max,
                                                 int32_t* status, int lane) {
  cut_starts(s.seg_start, offsets, groups, rows, status, lane);
  fill_schedule(s, s.seg_start, groups, rows, bn_max, lane);
}

// Warp-cooperative build of the schedule (called by one warp).
template <typename Problem>
__device__ __forceinline__ void build_schedule(SegSched& s, const Problem& a, int lane) {
  if (!fill_schedule(s, a.offsets, a.groups, a.rows, a.bn_max, lane))
    cut_schedule(s, a.offsets, a.groups, a.rows, a.bn_max, a.status, lane);
}
template <typename Problem>
__device__ __forceinline__ int total_tiles(const SegSched& s, const Problem& a) {
  return s.tb_start[a.groups] * a.n_mblk;
}

// a / b for 0 <= a, 0 < b: a float quotient where it is exact (a < 2^20: its
// error is below a quarter). Every role of a CTA decodes every tile, the loads'
// and the MMAs' threads between two tiles' work: integer divisions there cost a
// thousand cycles a tile.
__device__ __forceinline__ int quick_div(int a, int b) {
  return a < (1 << 20) ? __float2int_rz(__fdividef(static_cast<float>(a) + 0.5f, static_cast<float>(b))) : a / b;
}

// Tile `local` of a segment of n rows starting at row seg0 (group g).
template <typename Problem>
__device__ __forceinline__ SegTile decode_in_segment(const Problem& a, int g, int seg0, int n, int local) {
  SegTile ti;
  const int unit = seg_unit(a);
  ti.g = g;
  const int ntb = quick_div(n + a.bn_max - 1, a.bn_max);
  const int bn = (quick_div(n + ntb - 1, ntb) + unit - 1) & ~(unit - 1);
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
  ti.N = (ti.n_valid + unit - 1) & ~(unit - 1);
  return ti;
}
template <typename Problem>
__device__ __forceinline__ SegTile decode_in_group(const SegSched& s, const Problem& a, int g, int t) {
  return decode_in_segment(a, g, s.seg_start[g], s.seg_start[g + 1] - s.seg_start[g], t - s.tb_start[g] * a.n_mblk);
}

// Tile t; g: the group of the caller's last tile (0 at first; t only grows).
__device__ __forceinline__ SegTile decode_tile(const SegSched& s, const SegProblem& a, int t, int& g) {
  while (t >= s.tb_start[g + 1] * a.n_mblk) ++g;
  return decode_in_group(s, a, g, t);
}
// Tile t of a problem whose segments are the schedule's.
__device__ __forceinline__ SegTile decode_tile(const SegSched& s, const GemmArgs& a, int t) {
  int lo = 0, hi = a.groups - 1;   // last g whose first tile is no later than t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.tb_start[mid] * a.n_mblk <= t) lo = mid; else hi = mid - 1;
  }
  return decode_in_group(s, a, lo, t);
}

}  // namespace moe
