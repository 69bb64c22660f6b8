// Argument blocks and launchers of the microscaled 4-bit (MXFP4) kernels.
#pragma once

#include "kernels.cuh"

namespace moe {

// Pipeline stages of a 4-bit GEMM with tiles of bn rows.
constexpr int mx_stages(int bn) { return bn <= 64 ? 4 : 3; }

// A grouped GEMM of 4-bit weights and rows (K values a row, packed two a byte).
struct MxGemmArgs {
  int32_t rows = 0, K = 0, groups = 1;
  const int32_t* offsets = nullptr;    // [groups + 1] or nullptr (one segment)
  int32_t n_mblk = 0;                  // tiles of 256 weight rows per group
  int32_t bn_max = 32;                 // rows per tile at most: 32, 64 or 192
  int32_t stages = 4;                  // mx_stages(bn_max)
  const uint32_t* b_scale = nullptr;   // [K / 128, rows], four scale bytes each
  const float* row_w = nullptr;        // down: [rows] or nullptr
  void* out = nullptr;                 // gate/up: codes [rows, out_ld / 2]; down: bf16 [rows, out_ld]
  int32_t out_ld = 0;
  uint8_t* out_scale = nullptr;        // gate/up: [out_ld / 128, rows] words
  int32_t* status = nullptr;
  uint64_t wait_ns = kDefaultWaitLimitNs;
};
// What a stage loads, a box each: a block of 256 values (128 bytes) of K
constexpr int kMxRowBoxes = 12;
struct MxMaps {
  CUtensorMap w;                       // of 2 x 128 weight rows: gate and up of 128 features, or 256 rows of w2
  CUtensorMap w_scale;                 // their scales
  CUtensorMap rows[kMxRowBoxes];       // of 16 (i + 1) rows, up to bn_max
};
cudaError_t launch_mx_gemm(bool gate_up, const MxMaps& maps, const MxGemmArgs& a, int grid, cudaStream_t stream);
// src: row r of the result is row src[r] of a [a_rows, K] (nullptr: row r)
cudaError_t launch_mx_quant_rows(int rows, int K, const void* a, int a_rows, const int32_t* src, void* q, void* scale,
                                 int32_t* status, cudaStream_t stream);
cudaError_t launch_mx_dequant_rows(int rows, int K, const void* q, const void* scale, void* out, cudaStream_t stream);
cudaError_t launch_mx_quant_weights(int batch, int N, int K, const void* w, void* q, void* scale, cudaStream_t stream);

}  // namespace moe
