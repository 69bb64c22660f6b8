// Argument blocks and launchers of the training and the 4-bit kernels.
#pragma once

#include "kernels.cuh"

namespace moe {

// The training GEMMs over expert segments (train_gemm_kernel):
//   TRAIN_FORWARD  [g | u] = B w13^T, h = SiLU(g) * u; gu and h stored. K = H, M = I
//   TRAIN_HIDDEN   dh0 = B w2 (B = d_out), then the activation's backward. K = H, M = I
//   TRAIN_ROWS     out = B W (+ add), W [groups, K, M] row-major or tiled w13
enum { TRAIN_FORWARD = 0, TRAIN_HIDDEN = 1, TRAIN_ROWS = 2 };
struct TrainGemmArgs {
  int32_t rows = 0, K = 0, M = 0, groups = 1;
  const int32_t* offsets = nullptr;   // [groups + 1] or nullptr (one segment)
  int32_t n_mblk = 0;                 // feature blocks per group (set by the launcher)
  int32_t tiled = 0;                  // W in moe_tile_ffn_weights' layout
  __nv_bfloat16* gu = nullptr;        // [rows, 2I]: forward out, hidden in
  __nv_bfloat16* h = nullptr;         // [rows, I] out: forward h, hidden row_w * h
  const float* row_w = nullptr;       // hidden: [rows] or nullptr (= 1)
  __nv_bfloat16* d_gu = nullptr;      // hidden: [rows, 2I] out
  float* partial = nullptr;           // hidden: [I / 32, rows] out, partial sums of d_row_w
  int32_t parts = 1;                  // hidden: parts of K (hidden_parts; set by the launcher)
  __nv_bfloat16* out = nullptr;       // rows: [rows, M]
  const __nv_bfloat16* add = nullptr; // rows, one sub-tile: [rows, M] added to the product, or nullptr (may be `out`)
  int32_t* status = nullptr;
  uint64_t wait_ns = kDefaultWaitLimitNs;
};
// Half of a tile's token rows: box[i] has 16 (i + 1) rows.
struct HalfMaps {
  CUtensorMap box[8];
};
// Tiles of `feats` features x 256 rows at most: each segment that has rows adds
// at most one partial row block.
inline long long train_tiles(int rows, int groups, int M, int feats) {
  return (static_cast<long long>(rows) / 256 + (groups < rows ? groups : rows)) * ((M + feats - 1) / feats);
}
// Sub-tiles per CTA of a TRAIN_ROWS product of K terms (see train_gemm_kernel):
// two for a long K, where that leaves a tile for each pair of SMs. (48 rows on 8
// experts, K = 1280, 768 features: 16 tiles of 512 features, 13.6 us.)
inline int train_subs(int rows, int groups, int K, int M, int num_sms) {
  return K > 512 && train_tiles(rows, groups, M, 512) >= num_sms / 2 ? 2 : 1;
}
// Parts of K that dh0 is summed in, which are added up in fp32 with rounding: the
// tensor cores cut each of their sums towards zero, 16 terms at a time, and
// d_row_w, an fp32 output, is short with them (7168 terms of random rows in one
// sum: 7.9e-6 of its norm; equal signs lose up to three times as much). Parts of
// at most 896 terms lose 1.6e-6 at most, 9e-7 measured, for 1 to 2 % of a backward
// pass's time.
inline int hidden_parts(int K) { return (K + 895) / 896; }
cudaError_t launch_train_gemm(int mode, int subs, const CUtensorMap& tmA, const HalfMaps& tmB, const TrainGemmArgs& a,
                              int num_sms, cudaStream_t stream);
cudaError_t launch_row_w_grad(int rows, int n, const float* partial, const int32_t* offsets, int groups, float* d_row_w,
                              cudaStream_t stream);

// Weight gradients C[g] [M, N] = A[rows of g]^T B[rows of g]; up to two such
// products over the same segments in one launch.
struct WgradProblem {
  CUtensorMap tmA, tmB;               // [rows, M], [rows, N] bf16 as column blocks: 64 rows x 2 blocks of 64
  CUtensorMap tmOut;                  // [groups * M, N] bf16 or fp32, boxes of 32 rows x 128 bytes
  int32_t M, N, tiles;                // tiles = groups * per_group
  int32_t a_flat;                     // M % 64 != 0: tmA is the plain matrix, boxes of 64 rows x 64 columns
  int32_t per_group, m_blocks, n_blocks;   // tiles of a group; its blocks along M and N
};
struct WgradArgs {
  WgradProblem prob[2];
  int32_t n_prob, rows, groups;
  const int32_t* offsets;
  int32_t f32, accumulate;            // output type; fp32 only: add to what is there
  int32_t after, beside;              // launched behind a train_gemm_kernel it does not depend on, of so many tiles
  const float* partial;               // also d_row_w from its partial sums [n_partial, rows], or
  float* d_row_w;                     //   nullptr
  int32_t n_partial;
  int32_t* status;
  uint64_t wait_ns;
};
cudaError_t launch_wgrad(const WgradArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_route_backward(int T, int E, int k, int scoring, int norm, float scale, const float* logits,
                                  const int32_t* ids, const float* d_w, const int32_t* slot_to_row, float* d_logits,
                                  void* d_logits16, int32_t* status, cudaStream_t stream);

}  // namespace moe
