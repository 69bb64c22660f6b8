// C-ABI entry points of libmoe (declared in include/moe.h): argument checks on
// the host, TMA tensor-map encoding, kernel launches. No allocation happens
// here; every buffer belongs to the caller.
#include <atomic>
#include <initializer_list>
#include <mutex>

#include "mxfp4.cuh"
#include "train.cuh"


using namespace moe;

namespace {

thread_local int32_t g_last_cuda_error = 0;

moe_status cuda_fail(int32_t code) {
  g_last_cuda_error = code;
  return MOE_ERR_CUDA;
}

moe_status check_launch(cudaError_t e) {
  if (e != cudaSuccess) return cuda_fail(static_cast<int32_t>(e));
  return MOE_OK;
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

template <typename... P>
bool any_misaligned(P... ps) {
  return (misaligned(ps) || ...);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once through the runtime (so the
// library needs no link-time dependency on libcuda).
EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Encodes a tensor map of `ptr` (no interleaving, zeros outside, every element).
// The encoder wants the calling host thread's context, which a thread has only
// from its first runtime call that needs one: where there is none yet, it gets
// the current device's (allowed while a stream is captured).
moe_status encode(CUtensorMap* m, CUtensorMapDataType type, uint32_t rank, const void* ptr, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return cuda_fail(static_cast<int32_t>(cudaErrorNotSupported));
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  auto run = [&] {
    return enc(m, type, rank, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = run();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return cuda_fail(static_cast<int32_t>(e));
    r = run();
  }
  return r == CUDA_SUCCESS ? MOE_OK : cuda_fail(1000 + static_cast<int32_t>(r));
}

// Row-major [outer, inner] matrix; box = 128 bytes of `inner` x box_rows rows,
// 128-byte swizzle (the layout the tcgen05 smem descriptors expect).
moe_status make_tmap(CUtensorMap* m, const void* ptr, bool one_byte, uint64_t inner, uint64_t outer,
                     uint32_t box_rows) {
  const uint64_t esize = one_byte ? 1 : 2;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * esize};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / esize), box_rows};
  return encode(m, one_byte ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, dims, strides, box);
}

// Token-row maps of a grouped GEMM: bf16 rows are fetched with 256-, 128-,
// 64-, 32- and 16-row boxes; e4m3 rows (at most 32 tokens a tile) with one
// 32-row box.
moe_status make_token_tmaps(TokenMaps* m, const void* ptr, bool fp8, uint64_t K, uint64_t rows) {
  if (fp8) return make_tmap(&m->box[0], ptr, true, K, rows, 32);
  for (int i = 0; i < kTokBoxes; ++i) {
    moe_status s = make_tmap(&m->box[i], ptr, false, K, rows, 256u >> i);
    if (s != MOE_OK) return s;
  }
  return MOE_OK;
}

// A 3-D bf16 tensor map with 128-byte swizzle; strides in bytes.
moe_status make_tmap_3d(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1, uint64_t s2,
                        uint32_t b1, uint32_t b2) {
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {s1, s2};
  cuuint32_t box[3] = {64, b1, b2};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, dims, strides, box);
}

// A row-major bf16 matrix [rows, cols] as [cols / 64] blocks of [rows, 64];
// boxes of 64 rows of `blocks` blocks.
moe_status make_block_tmap(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint32_t blocks = 2) {
  return make_tmap_3d(m, ptr, 64, rows, cols / 64, cols * 2, 128, 64, blocks);
}

// A weight as train_gemm_kernel loads it, one box per block of 64 K:
//   forward (w13 [groups, 2, I, H]): 128 gate rows and the same features' up
//     rows; tiled: one 256-row block.
//   else ([groups, K, M] or its tiled copy, K blocks of 256 rows): 64 K rows x
//     128 * subs features, as column blocks of 64.
moe_status make_train_weight_tmap(CUtensorMap* m, const void* w, int mode, int tiled, int64_t groups, int64_t K, int64_t M,
                                  int subs) {
  if (tiled) {
    const uint64_t values = static_cast<uint64_t>(groups) * K * M * (mode == TRAIN_FORWARD ? 2 : 1);
    return make_tmap_3d(m, w, 64, 256, values / (64 * 256), 128, 256 * 128, mode == TRAIN_FORWARD ? 256 : 64,
                        mode == TRAIN_FORWARD ? 1 : 2 * subs);
  }
  if (mode == TRAIN_FORWARD) return make_tmap_3d(m, w, K, M, 2 * groups, K * 2, K * 2 * M, 128, 2);
  return make_block_tmap(m, w, M, groups * K, 2 * subs);
}

// Token-row maps of a CTA pair: one box for each half tile of 16, 32, .. 128
// rows that can occur: up to half of `rows`, or, with one segment of all rows
// (no offsets), those of its full tiles and of its last one. The others are
// copies, never loaded with.
moe_status make_half_tmaps(HalfMaps* m, const void* ptr, uint64_t K, int32_t rows, const int32_t* offsets) {
  const int32_t blocks = (rows + 255) / 256;
  const int32_t full = ((rows + blocks - 1) / blocks + 31) / 32, last = (rows - (blocks - 1) * 32 * full + 31) / 32;
  const int32_t most = blocks > 1 ? 8 : (rows + 31) / 32;
  int32_t made = -1;
  for (int32_t i = 0; i < 8; ++i) {
    if (offsets ? i >= most : i + 1 != full && i + 1 != last) continue;
    moe_status s = make_tmap(&m->box[i], ptr, false, K, static_cast<uint64_t>(rows), 16 * (i + 1));
    if (s != MOE_OK) return s;
    if (made < 0)
      for (int32_t j = 0; j < i; ++j) m->box[j] = m->box[i];
    made = i;
    for (int32_t j = i + 1; j < 8; ++j) m->box[j] = m->box[i];
  }
  return MOE_OK;
}

moe_status sm_count(int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e);
  return MOE_OK;
}

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// Limit of every bounded device-side wait, passed to the kernels at launch
// (moe_set_wait_limit_ns; 2 s unless changed).
std::atomic<uint64_t> g_wait_limit_ns{kDefaultWaitLimitNs};
uint64_t wait_limit() { return g_wait_limit_ns.load(std::memory_order_relaxed); }

}  // namespace

extern "C" {

int32_t moe_abi_version(void) { return MOE_ABI_VERSION; }

int32_t moe_last_cuda_error(void) { return g_last_cuda_error; }

moe_status moe_set_wait_limit_ns(uint64_t ns) {
  g_wait_limit_ns.store(ns == 0 ? kDefaultWaitLimitNs : ns, std::memory_order_relaxed);
  return MOE_OK;
}

uint64_t moe_wait_limit_ns(void) { return wait_limit(); }

const char* moe_status_string(moe_status s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case MOE_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
    case MOE_ERR_CUDA: return "CUDA error";
    case MOE_ERR_DEVICE_CHECK: return "device-side bounds check failed";
    case MOE_ERR_DEVICE_TIMEOUT: return "device-side bounded wait timed out";
    default: return "unknown status";
  }
}

// logits = x @ gate^T on the clustered gate GEMM (r carries T, H, E, logits,
// status), and with `route` the routing of every token in the same launch
moe_status gate_gemm(const RouteArgs& r, const void* x, const void* gate_w, bool route, int nsm, cudaStream_t st) {
  CUtensorMap tmX, tmG;
  moe_status s = make_tmap(&tmX, x, false, r.H, r.T, 128);
  if (s != MOE_OK) return s;
  s = make_tmap(&tmG, gate_w, false, r.H, r.E, static_cast<uint32_t>(r.E));
  if (s != MOE_OK) return s;
  return check_launch(launch_gate_gemm(tmX, tmG, r, route, nsm, st));
}

moe_status moe_gate_logits(int32_t T, int32_t H, int32_t E, const void* x, const void* gate_w, float* logits,
                           int32_t* dev_status, void* stream) {
  if (T < 1 || H < 64 || !x || !gate_w || !logits) return MOE_ERR_INVALID_ARG;
  if (H % 64 != 0 || E > 256 || E < 16 || E % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(x, gate_w, logits)) return MOE_ERR_ALIGNMENT;
  int nsm = 0;
  moe_status s = sm_count(&nsm);
  if (s != MOE_OK) return s;
  RouteArgs r{};
  r.T = T;
  r.H = H;
  r.E = E;
  r.logits = logits;
  r.status = dev_status;
  r.wait_ns = wait_limit();
  return gate_gemm(r, x, gate_w, false, nsm, as_stream(stream));
}

moe_status moe_route(const moe_route_params* p, const void* x, const void* gate_w, const float* sel_bias,
                     float* logits, int32_t* topk_ids, float* topk_w, int32_t* expert_counts, void* stream) {
  if (!p || !topk_ids || !topk_w || !expert_counts || !logits) return MOE_ERR_INVALID_ARG;
  if (p->T < 1 || p->k < 1 || p->n_group < 1 || p->topk_group < 1) return MOE_ERR_INVALID_ARG;
  if (p->scoring != MOE_SOFTMAX && p->scoring != MOE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (p->E < 1 || p->E % p->n_group != 0 || p->topk_group > p->n_group) return MOE_ERR_INVALID_ARG;
  if (p->k > p->topk_group * (p->E / p->n_group)) return MOE_ERR_INVALID_ARG;
  if (p->k > 16 || p->E > 256 || p->E < 16 || p->E % 16 != 0 || p->n_group > 32) return MOE_ERR_UNSUPPORTED;
  if (x) {
    if (!gate_w || p->H < 64) return MOE_ERR_INVALID_ARG;
    if (p->H % 64 != 0) return MOE_ERR_UNSUPPORTED;
  }
  if (any_misaligned(x, gate_w, sel_bias, logits, topk_ids, topk_w, expert_counts)) return MOE_ERR_ALIGNMENT;
  int nsm = 0;
  moe_status s = sm_count(&nsm);
  if (s != MOE_OK) return s;
  cudaStream_t st = as_stream(stream);
  RouteArgs r{p->T, p->H, p->E, p->k, p->n_group, p->topk_group, p->scoring, p->norm_topk_prob ? 1 : 0,
              p->routed_scaling_factor, sel_bias, logits, topk_ids, topk_w, expert_counts, p->dev_status,
              wait_limit()};
  cudaError_t e = cudaMemsetAsync(expert_counts, 0, sizeof(int32_t) * p->E, st);
  if (e != cudaSuccess) return cuda_fail(e);
  // from x: one launch (projection + routing) where the shape allows
  if (x) {
    const bool fused = route8_experts_per_thread(r) > 0;
    if ((s = gate_gemm(r, x, gate_w, fused, nsm, st)) != MOE_OK) return s;
    if (fused) return MOE_OK;
  }
  return check_launch(launch_route_tokens(r, nsm, st));
}

moe_status moe_permute_workspace_size(int32_t T, int32_t k, int32_t E, size_t* bytes) {
  if (!bytes || T < 1 || k < 1 || E < 1) return MOE_ERR_INVALID_ARG;
  *bytes = permute_workspace_bytes(T, E);
  return MOE_OK;
}

moe_status moe_permute(int32_t T, int32_t k, int32_t E, int32_t H, const int32_t* topk_ids,
                       const float* topk_w, const void* x, moe_dtype x_dtype, const float* x_scale,
                       void* x_perm, moe_dtype perm_dtype, float* x_perm_scale, void* x_q, float* x_q_scale,
                       int32_t* expert_offsets, int32_t* src_token, int32_t* slot_to_row, float* row_w,
                       void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (T < 1 || k < 1 || E < 1 || H < 1 || k > E) return MOE_ERR_INVALID_ARG;
  if (!topk_ids || !expert_offsets || !src_token || !slot_to_row || !workspace) return MOE_ERR_INVALID_ARG;
  if (row_w && !topk_w) return MOE_ERR_INVALID_ARG;
  if ((x_perm || x_q) && !x) return MOE_ERR_INVALID_ARG;
  if (x_dtype != MOE_BF16 && x_dtype != MOE_E4M3) return MOE_ERR_INVALID_ARG;
  if (perm_dtype != MOE_BF16 && perm_dtype != MOE_E4M3) return MOE_ERR_INVALID_ARG;
  if (x_dtype == MOE_E4M3 && perm_dtype != MOE_E4M3) return MOE_ERR_UNSUPPORTED;
  const bool quant = x_dtype == MOE_BF16 && perm_dtype == MOE_E4M3;
  if ((x_q || x_q_scale) && (!quant || !x_q || !x_q_scale)) return MOE_ERR_INVALID_ARG;
  if (k > 16 || E > 1024) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(T) * k > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  if (perm_dtype == MOE_BF16) {
    if (H % 8 != 0) return MOE_ERR_UNSUPPORTED;
  } else {
    if (H % 128 != 0) return MOE_ERR_UNSUPPORTED;
    if (x_perm && !x_perm_scale) return MOE_ERR_INVALID_ARG;
    if (x_dtype == MOE_E4M3 && x_perm && !x_scale) return MOE_ERR_INVALID_ARG;
  }
  if (workspace_bytes < permute_workspace_bytes(T, E)) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(topk_ids, topk_w, x, x_scale, x_perm, x_perm_scale, x_q, x_q_scale, expert_offsets,
                     src_token, slot_to_row, row_w, workspace))
    return MOE_ERR_ALIGNMENT;
  return check_launch(launch_permute(T, k, E, H, x_dtype == MOE_E4M3, perm_dtype == MOE_E4M3, topk_ids, topk_w, x,
                                     x_scale, x_perm, x_perm_scale, x_q, x_q_scale, expert_offsets, src_token,
                                     slot_to_row, row_w, static_cast<int32_t*>(workspace), dev_status,
                                     as_stream(stream)));
}

}  // extern "C"

namespace {

// Memory a call reads or writes (ptr may be nullptr), and whether its outputs
// overlap neither an input nor one another.
struct Span {
  const void* ptr;
  size_t bytes;
};
Span offsets_span(const int32_t* offsets, int32_t groups) { return {offsets, (static_cast<size_t>(groups) + 1) * 4}; }
bool overlap(const Span& p, const Span& q) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p.ptr), b = reinterpret_cast<uintptr_t>(q.ptr);
  return p.ptr && q.ptr && a < b + q.bytes && b < a + p.bytes;
}
bool outputs_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (overlap(*o, i)) return false;
    for (auto n = o + 1; n != outs.end(); ++n)
      if (overlap(*o, *n)) return false;
  }
  return true;
}

// Shared checks of the grouped SwiGLU calls; `a` is the GEMM's activation
// operand (x for the first GEMM, h for the second).
moe_status check_ffn(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* a,
                     const float* a_scale, bool need_w13, bool need_w2) {
  if (!w || !a) return MOE_ERR_INVALID_ARG;
  if ((need_w13 && !w->w13) || (need_w2 && !w->w2)) return MOE_ERR_INVALID_ARG;
  if (rows < 1 || H < 1 || w->I < 1 || w->groups < 1) return MOE_ERR_INVALID_ARG;
  if (w->dtype != MOE_BF16 && w->dtype != MOE_E4M3 && w->dtype != MOE_MXFP4) return MOE_ERR_INVALID_ARG;
  if (w->tiled != 0 && w->tiled != 1) return MOE_ERR_INVALID_ARG;
  if (w->tiled && w->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (H % 256 != 0 || w->I % 128 != 0 || w->groups > 512) return MOE_ERR_UNSUPPORTED;
  if (w->dtype != MOE_BF16 && ((need_w13 && !w->w13_scale) || (need_w2 && !w->w2_scale) || !a_scale))
    return MOE_ERR_INVALID_ARG;
  if (w->dtype == MOE_E4M3) {
    if (H > 8192 || w->I > 8192) return MOE_ERR_UNSUPPORTED;
  }
  if (static_cast<long long>(w->groups) * 2 * w->I > 0x7fffffffLL ||
      static_cast<long long>(w->groups) * H > 0x7fffffffLL)
    return MOE_ERR_UNSUPPORTED;
  // the tiled view's rows are TMA coordinates (int32)
  if (w->tiled && static_cast<long long>(w->groups) * 2 * w->I * (H / 64) > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(w->w13, w->w2, w->w13_scale, w->w2_scale, a, a_scale)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// Token blocks (of at most 256 rows) of `rows` rows in one segment, and an
// upper bound over `groups` segments of `rows` rows in all (each non-empty
// segment adds at most one partial block).
int32_t ffn_blocks(int32_t rows) { return (rows + 255) / 256; }
int32_t ffn_routed_blocks(int32_t rows, int32_t groups) { return ffn_blocks(rows) + groups; }

// Tensor maps and kernel arguments of one grouped GEMM.
struct GemmPlan {
  CUtensorMap tmA;
  TokenMaps tmB;
  GemmArgs g;
  bool fp8;
};

// Kernel choice for the bf16 grouped GEMMs, by measurement at the V3 shape on
// B200: single CTAs, 256-token tiles with one TMEM accumulator pair, three
// 64-K stages; 4 epilogue warps for gate/up and 12 for down, whose output
// rows are twice as wide (three warps per TMEM lane quarter take turns on
// its 32-token chunks). E4M3: at most 32 tokens a tile.
moe_status plan_gate_up(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* a, const float* a_scale,
                        const int32_t* offsets, void* h_ws, float* h_scale_ws, int32_t* dev_status, GemmPlan* p) {
  const bool fp8 = w->dtype == MOE_E4M3;
  const int I = w->I;
  // tiled weights: a [*, 64] matrix whose 256-row boxes (128 gate rows, then
  // the same features' 128 up rows) are the tiles
  moe_status s = w->tiled ? make_tmap(&p->tmA, w->w13, false, 64, static_cast<uint64_t>(w->groups) * 2 * I * (H / 64), 256)
                          : make_tmap(&p->tmA, w->w13, fp8, H, static_cast<uint64_t>(w->groups) * 2 * I, 128);
  if (s != MOE_OK) return s;
  if ((s = make_token_tmaps(&p->tmB, a, fp8, H, rows)) != MOE_OK) return s;
  GemmArgs& g = p->g;
  g = GemmArgs{};
  g.rows = rows;
  g.K = H;
  g.groups = w->groups;
  g.offsets = offsets;
  g.a_rows_per_group = 2 * I;            // w13[e]: gate rows [0, I), up rows [I, 2I)
  g.a_tiled = w->tiled;
  g.n_mblk = I / 128;
  g.mblk_stride = 128;
  g.sub1_off = I;                        // sub-tile 1: the up rows of the same 128 features
  g.feat_stride = 128;
  g.bn_max = fp8 ? 32 : 256;
  g.out = h_ws;
  g.out_ld = I;
  g.a_scale = w->w13_scale;
  g.b_scale = a_scale;
  g.out_scale = h_scale_ws;
  g.status = dev_status;
  g.epi_warps = 4;
  g.wait_ns = wait_limit();
  p->fp8 = fp8;
  return MOE_OK;
}

moe_status plan_down(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* h, const float* h_scale,
                     const int32_t* offsets, const float* row_w, void* out, int32_t* dev_status, GemmPlan* p) {
  const bool fp8 = w->dtype == MOE_E4M3;
  const int I = w->I;
  // bf16: a tile's 256 contiguous w2 rows are one TMA box
  moe_status s = w->tiled ? make_tmap(&p->tmA, w->w2, false, 64, static_cast<uint64_t>(w->groups) * H * (I / 64), 256)
                          : make_tmap(&p->tmA, w->w2, fp8, I, static_cast<uint64_t>(w->groups) * H, fp8 ? 128 : 256);
  if (s != MOE_OK) return s;
  if ((s = make_token_tmaps(&p->tmB, h, fp8, I, rows)) != MOE_OK) return s;
  GemmArgs& g = p->g;
  g = GemmArgs{};
  g.rows = rows;
  g.K = I;
  g.groups = w->groups;
  g.offsets = offsets;
  g.a_rows_per_group = H;
  g.a_tiled = w->tiled;
  g.n_mblk = H / 256;
  g.mblk_stride = 256;
  g.sub1_off = 128;                      // sub-tiles: w2 rows [mb*256, +128) and [mb*256 + 128, +128)
  g.feat_stride = 256;
  g.feat_sub1 = 128;
  g.bn_max = fp8 ? 32 : 256;
  g.a_one_box = fp8 ? 0 : 1;
  g.out = out;
  g.out_ld = H;
  g.row_w = row_w;
  g.a_scale = w->w2_scale;
  g.b_scale = h_scale;
  g.status = dev_status;
  g.epi_warps = 12;
  g.wait_ns = wait_limit();
  p->fp8 = fp8;
  return MOE_OK;
}

moe_status launch_plan(const GemmPlan& p, int epi, cudaStream_t st, int nsm, const GemmPlan* second = nullptr) {

  // one launch needs the same kernel form for both: bf16, same tile shape
  const bool one = second && !p.fp8 && !second->fp8 && p.g.bn_max == second->g.bn_max &&
                   p.g.epi_warps == second->g.epi_warps;
  if (second && !one) {
    moe_status s = check_launch(launch_grouped_gemm(p.fp8, epi, p.tmA, p.tmB, p.g, nsm, st));
    return s != MOE_OK ? s : check_launch(launch_grouped_gemm(second->fp8, epi, second->tmA, second->tmB,
                                                              second->g, nsm, st));
  }
  if (!second) return check_launch(launch_grouped_gemm(p.fp8, epi, p.tmA, p.tmB, p.g, nsm, st));
  const SecondProblem two{second->tmA, second->tmB, second->g};
  return check_launch(launch_grouped_gemm(p.fp8, epi, p.tmA, p.tmB, p.g, nsm, st, &two));
}

// Rows per tile and pipeline stages of the 4-bit GEMMs, by the rows an expert
// has on average. A small tile leaves room for more stages of weights in flight,
// which is what counts at a few rows per expert; twice the average, so that most
// segments still fit one tile and their weights are read once.
void mx_tile(int32_t rows, int32_t groups, MxGemmArgs* g) {
  const int32_t twice = 2 * ((rows + groups - 1) / groups);
  g->bn_max = twice <= 32 ? 32 : twice <= 64 ? 64 : 192;
  g->stages = mx_stages(g->bn_max);
}

// A 4-bit weight's codes, w13 as [2 groups][I] rows (a gate block and the same
// features' up block lie I rows apart), w2 as [groups * H / 128][128], in boxes of
// 2 x 128 rows of 128 bytes; its scales, 512 bytes per 128 x 128 values, in boxes
// of the same 256 rows x 256 values.
moe_status make_mx_weight_tmaps(MxMaps* m, bool gate_up, const moe_ffn_weights* w, int32_t H) {
  const uint64_t K = gate_up ? H : w->I, n = gate_up ? w->I : 128;
  const uint64_t blocks = gate_up ? 2 * static_cast<uint64_t>(w->groups) : static_cast<uint64_t>(w->groups) * (H / 128);
  cuuint64_t dims[3] = {K / 2, n, blocks}, strides[2] = {K / 2, K / 2 * n};
  cuuint32_t box[3] = {128, 128, 2};
  moe_status s = encode(&m->w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, gate_up ? w->w13 : w->w2, dims, strides, box);
  if (s != MOE_OK) return s;
  const uint64_t kb = K / 128, sn = gate_up ? w->I / 128 : blocks, sb = gate_up ? blocks : 1;
  cuuint64_t sdims[4] = {128, kb, sn, sb}, sstrides[3] = {512, 512 * kb, 512 * kb * sn};
  cuuint32_t sbox[4] = {128, 2, gate_up ? 1u : 2u, gate_up ? 2u : 1u};
  return encode(&m->w_scale, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, gate_up ? w->w13_scale : w->w2_scale, sdims, sstrides, sbox,
                CU_TENSOR_MAP_SWIZZLE_NONE);
}

// One 4-bit grouped GEMM (scales as moe_quantize_mxfp4_rows / _weights lay them out).
moe_status run_mx(bool gate_up, int32_t rows, int32_t H, const moe_ffn_weights* w, const void* act, const void* act_scale,
                  const int32_t* offsets, const float* row_w, void* out, void* out_scale, int32_t* dev_status,
                  cudaStream_t st, int nsm) {
  const int32_t I = w->I, K = gate_up ? H : I;
  MxGemmArgs g;
  g.rows = rows;
  g.K = K;
  g.groups = w->groups;
  g.offsets = offsets;
  g.n_mblk = gate_up ? I / 128 : H / 256;
  mx_tile(rows, w->groups, &g);
  g.b_scale = static_cast<const uint32_t*>(act_scale);
  g.row_w = row_w;
  g.out = out;
  g.out_ld = gate_up ? I : H;
  g.out_scale = static_cast<uint8_t*>(out_scale);
  g.status = dev_status;
  g.wait_ns = wait_limit();
  MxMaps m;
  moe_status s = make_mx_weight_tmaps(&m, gate_up, w, H);
  if (s != MOE_OK) return s;
  for (int i = 0; i < g.bn_max / 16; ++i)
    if ((s = make_tmap(&m.rows[i], act, true, K / 2, rows, 16 * (i + 1))) != MOE_OK) return s;
  return check_launch(launch_mx_gemm(gate_up, m, g, nsm, st));
}

moe_status run_gate_up(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* a,
                       const float* a_scale, const int32_t* offsets, void* h_ws, float* h_scale_ws,
                       int32_t* dev_status, cudaStream_t st, int nsm) {
  if (w->dtype == MOE_MXFP4)
    return run_mx(true, rows, H, w, a, a_scale, offsets, nullptr, h_ws, h_scale_ws, dev_status, st, nsm);
  GemmPlan p;
  moe_status s = plan_gate_up(rows, H, w, a, a_scale, offsets, h_ws, h_scale_ws, dev_status, &p);
  return s != MOE_OK ? s : launch_plan(p, EPI_SWIGLU, st, nsm);
}

moe_status run_down(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* h, const float* h_scale,
                    const int32_t* offsets, const float* row_w, void* out, int32_t* dev_status,
                    cudaStream_t st, int nsm) {
  if (w->dtype == MOE_MXFP4)
    return run_mx(false, rows, H, w, h, h_scale, offsets, row_w, out, nullptr, dev_status, st, nsm);
  GemmPlan p;
  moe_status s = plan_down(rows, H, w, h, h_scale, offsets, row_w, out, dev_status, &p);
  return s != MOE_OK ? s : launch_plan(p, EPI_WEIGHTED, st, nsm);
}


}  // namespace

extern "C" {

moe_status moe_gate_up_swiglu(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* a,
                              const float* a_scale, const int32_t* offsets, void* h_ws, float* h_scale_ws,
                              int32_t* dev_status, void* stream) {
  moe_status s = check_ffn(rows, H, w, a, a_scale, true, false);
  if (s != MOE_OK) return s;
  if (!h_ws || (!offsets && w->groups != 1)) return MOE_ERR_INVALID_ARG;
  if (w->dtype != MOE_BF16 && !h_scale_ws) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(offsets, h_ws, h_scale_ws)) return MOE_ERR_ALIGNMENT;
  int nsm = 0;
  if ((s = sm_count(&nsm)) != MOE_OK) return s;
  return run_gate_up(rows, H, w, a, a_scale, offsets, h_ws, h_scale_ws, dev_status, as_stream(stream), nsm);
}

moe_status moe_gate_up_swiglu_gather(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* x, int32_t T,
                                     const int32_t* src_token, const int32_t* offsets, void* h_ws,
                                     int32_t* dev_status, void* stream) {
  moe_status s = check_ffn(rows, H, w, x, nullptr, true, false);
  if (s != MOE_OK) return s;
  if (w->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (T < 1 || !src_token || !offsets || !h_ws) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(src_token, offsets, h_ws)) return MOE_ERR_ALIGNMENT;
  int nsm = 0;
  if ((s = sm_count(&nsm)) != MOE_OK) return s;
  const int I = w->I;
  CUtensorMap tmA;
  TokenMaps tmB;
  s = w->tiled ? make_tmap(&tmA, w->w13, false, 64, static_cast<uint64_t>(w->groups) * 2 * I * (H / 64), 256)
               : make_tmap(&tmA, w->w13, false, H, static_cast<uint64_t>(w->groups) * 2 * I, 128);
  if (s != MOE_OK) return s;
  s = make_token_tmaps(&tmB, x, false, H, T);      // not read: token rows are gathered
  if (s != MOE_OK) return s;
  GemmArgs g1{};
  g1.rows = rows;
  g1.K = H;
  g1.groups = w->groups;
  g1.offsets = offsets;
  g1.a_rows_per_group = 2 * I;
  g1.a_tiled = w->tiled;
  g1.n_mblk = I / 128;
  g1.mblk_stride = 128;
  g1.sub1_off = I;
  g1.feat_stride = 128;
  g1.out = h_ws;
  g1.out_ld = I;
  g1.status = dev_status;
  g1.gather_src = x;
  g1.gather_rows = src_token;
  g1.gather_src_rows = T;
  g1.wait_ns = wait_limit();
  return check_launch(launch_grouped_gemm(false, EPI_SWIGLU, tmA, tmB, g1, nsm, as_stream(stream)));
}

moe_status moe_gate_up_swiglu_train(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* a,
                                    const int32_t* offsets, void* h, void* gu, int32_t* dev_status, void* stream) {
  moe_status s = check_ffn(rows, H, w, a, nullptr, true, false);
  if (s != MOE_OK) return s;
  if (w->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (!h || !gu || (!offsets && w->groups != 1)) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(offsets, h, gu)) return MOE_ERR_ALIGNMENT;
  const int I = w->I;
  const size_t r = static_cast<size_t>(rows);
  if (!outputs_apart({{h, r * I * 2}, {gu, r * I * 4}}, {{a, r * H * 2}, {w->w13, static_cast<size_t>(w->groups) * I * H * 4},
                                                         offsets_span(offsets, w->groups)}))
    return MOE_ERR_INVALID_ARG;
  int nsm = 0;
  if ((s = sm_count(&nsm)) != MOE_OK) return s;
  CUtensorMap tmA;
  HalfMaps tmB;
  s = make_train_weight_tmap(&tmA, w->w13, TRAIN_FORWARD, w->tiled, w->groups, H, I, 2);
  if (s != MOE_OK) return s;
  if ((s = make_half_tmaps(&tmB, a, H, rows, offsets)) != MOE_OK) return s;
  TrainGemmArgs g;
  g.rows = rows;
  g.K = H;
  g.M = I;
  g.groups = w->groups;
  g.offsets = offsets;
  g.tiled = w->tiled;
  g.gu = static_cast<__nv_bfloat16*>(gu);
  g.h = static_cast<__nv_bfloat16*>(h);
  g.status = dev_status;
  g.wait_ns = wait_limit();
  return check_launch(launch_train_gemm(TRAIN_FORWARD, 2, tmA, tmB, g, nsm, as_stream(stream)));
}

moe_status moe_down_proj(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* h, const float* h_scale,
                         const int32_t* offsets, const float* row_w, void* out, int32_t* dev_status,
                         void* stream) {
  moe_status s = check_ffn(rows, H, w, h, h_scale, false, true);
  if (s != MOE_OK) return s;
  if (!out || (!offsets && w->groups != 1)) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(offsets, row_w, out)) return MOE_ERR_ALIGNMENT;
  int nsm = 0;
  if ((s = sm_count(&nsm)) != MOE_OK) return s;
  return run_down(rows, H, w, h, h_scale, offsets, row_w, out, dev_status, as_stream(stream), nsm);
}

moe_status moe_grouped_swiglu(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* a,
                              const float* a_scale, const int32_t* offsets, const float* row_w,
                              void* h_ws, float* h_scale_ws, void* out, int32_t* dev_status, void* stream) {
  moe_status s = check_ffn(rows, H, w, a, a_scale, true, true);
  if (s != MOE_OK) return s;
  if (!h_ws || !out || (!offsets && w->groups != 1)) return MOE_ERR_INVALID_ARG;
  if (w->dtype != MOE_BF16 && !h_scale_ws) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(offsets, row_w, h_ws, h_scale_ws, out)) return MOE_ERR_ALIGNMENT;
  int nsm = 0;
  if ((s = sm_count(&nsm)) != MOE_OK) return s;
  cudaStream_t st = as_stream(stream);
  s = run_gate_up(rows, H, w, a, a_scale, offsets, h_ws, h_scale_ws, dev_status, st, nsm);
  if (s != MOE_OK) return s;
  return run_down(rows, H, w, h_ws, h_scale_ws, offsets, row_w, out, dev_status, st, nsm);
}

moe_status moe_gate_up_swiglu_with_shared(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* a,
                                          const float* a_scale, const int32_t* offsets, void* h_ws,
                                          float* h_scale_ws, int32_t sh_rows, const moe_ffn_weights* sw,
                                          const void* sh_a, const float* sh_a_scale, void* sh_h_ws,
                                          float* sh_h_scale_ws, int32_t* dev_status, void* stream) {
  moe_status s = check_ffn(rows, H, w, a, a_scale, true, false);
  if (s != MOE_OK) return s;
  if ((s = check_ffn(sh_rows, H, sw, sh_a, sh_a_scale, true, false)) != MOE_OK) return s;
  if (!offsets || !h_ws || !sh_h_ws || sw->groups != 1 || sw->dtype != w->dtype) return MOE_ERR_INVALID_ARG;
  if (w->dtype != MOE_BF16 && (!h_scale_ws || !sh_h_scale_ws)) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(offsets, h_ws, h_scale_ws, sh_h_ws, sh_h_scale_ws)) return MOE_ERR_ALIGNMENT;
  int nsm = 0;
  if ((s = sm_count(&nsm)) != MOE_OK) return s;
  cudaStream_t st = as_stream(stream);
  if (w->dtype == MOE_MXFP4) {
    s = run_gate_up(rows, H, w, a, a_scale, offsets, h_ws, h_scale_ws, dev_status, st, nsm);
    return s != MOE_OK ? s : run_gate_up(sh_rows, H, sw, sh_a, sh_a_scale, nullptr, sh_h_ws, sh_h_scale_ws, dev_status, st, nsm);
  }
  GemmPlan p, q;
  if ((s = plan_gate_up(rows, H, w, a, a_scale, offsets, h_ws, h_scale_ws, dev_status, &p)) != MOE_OK) return s;
  if ((s = plan_gate_up(sh_rows, H, sw, sh_a, sh_a_scale, nullptr, sh_h_ws, sh_h_scale_ws, dev_status, &q)) !=
      MOE_OK)
    return s;
  return launch_plan(p, EPI_SWIGLU, st, nsm, &q);
}

moe_status moe_down_proj_with_shared(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* h,
                                     const float* h_scale, const int32_t* offsets, const float* row_w, void* out,
                                     int32_t sh_rows, const moe_ffn_weights* sw, const void* sh_h,
                                     const float* sh_h_scale, void* sh_out, int32_t* dev_status, void* stream) {
  moe_status s = check_ffn(rows, H, w, h, h_scale, false, true);
  if (s != MOE_OK) return s;
  if ((s = check_ffn(sh_rows, H, sw, sh_h, sh_h_scale, false, true)) != MOE_OK) return s;
  if (!offsets || !out || !sh_out || sw->groups != 1 || sw->dtype != w->dtype) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(offsets, row_w, out, sh_out)) return MOE_ERR_ALIGNMENT;
  int nsm = 0;
  if ((s = sm_count(&nsm)) != MOE_OK) return s;
  cudaStream_t st = as_stream(stream);
  if (w->dtype == MOE_MXFP4) {
    s = run_down(rows, H, w, h, h_scale, offsets, row_w, out, dev_status, st, nsm);
    return s != MOE_OK ? s : run_down(sh_rows, H, sw, sh_h, sh_h_scale, nullptr, nullptr, sh_out, dev_status, st, nsm);
  }
  GemmPlan p, q;
  if ((s = plan_down(rows, H, w, h, h_scale, offsets, row_w, out, dev_status, &p)) != MOE_OK) return s;
  if ((s = plan_down(sh_rows, H, sw, sh_h, sh_h_scale, nullptr, nullptr, sh_out, dev_status, &q)) != MOE_OK)
    return s;
  return launch_plan(p, EPI_WEIGHTED, st, nsm, &q);
}

moe_status moe_tile_ffn_weights(int32_t H, const moe_ffn_weights* src, void* w13_t, void* w2_t, void* stream) {
  if (!src || H < 1 || src->groups < 1 || src->I < 1 || src->tiled != 0) return MOE_ERR_INVALID_ARG;
  if (src->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (H % 256 != 0 || src->I % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(src->groups) * 2 * src->I * (H / 64) > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  if ((w13_t && !src->w13) || (w2_t && !src->w2)) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(src->w13, src->w2, w13_t, w2_t)) return MOE_ERR_ALIGNMENT;
  // the copies are gathers: an output overlapping any input would be read after being written
  const size_t b13 = static_cast<size_t>(src->groups) * 2 * src->I * H * 2, b2 = static_cast<size_t>(src->groups) * H * src->I * 2;
  if (!outputs_apart({{w13_t, b13}, {w2_t, b2}}, {{src->w13, b13}, {src->w2, b2}})) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = as_stream(stream);
  if (w13_t) {   // 256-row tiles: 128 gate rows, then the same features' 128 up rows
    moe_status s = check_launch(launch_tile_weights(src->w13, w13_t, src->groups, 2 * src->I, H, src->I, st));
    if (s != MOE_OK) return s;
  }
  if (w2_t) return check_launch(launch_tile_weights(src->w2, w2_t, src->groups, H, src->I, 0, st));
  return MOE_OK;
}

moe_status moe_swiglu_ffn_sync_size(int32_t rows, int32_t groups, int32_t sh_rows, size_t* bytes) {
  if (!bytes || rows < 1 || groups < 1 || sh_rows < 1) return MOE_ERR_INVALID_ARG;
  *bytes = sizeof(int32_t) * (ffn_routed_blocks(rows, groups) + ffn_blocks(sh_rows) + 1);
  return MOE_OK;
}

moe_status moe_swiglu_ffn_with_shared(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* a,
                                      const int32_t* offsets, const float* row_w, void* h_ws, void* out,
                                      int32_t sh_rows, const moe_ffn_weights* sw, const void* sh_a, void* sh_h_ws,
                                      void* sh_out, void* sync_ws, size_t sync_ws_bytes, int32_t* dev_status,
                                      void* stream) {
  moe_status s = check_ffn(rows, H, w, a, nullptr, true, true);
  if (s != MOE_OK) return s;
  if ((s = check_ffn(sh_rows, H, sw, sh_a, nullptr, true, true)) != MOE_OK) return s;
  if (!offsets || !h_ws || !out || !sh_h_ws || !sh_out || !sync_ws || sw->groups != 1) return MOE_ERR_INVALID_ARG;
  if (w->dtype != MOE_BF16 || sw->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  const size_t nctr = ffn_routed_blocks(rows, w->groups) + ffn_blocks(sh_rows);
  const size_t need = sizeof(int32_t) * (nctr + 1);   // token-block counters, then the tile counter
  if (sync_ws_bytes < need) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(offsets, row_w, h_ws, out, sh_h_ws, sh_out, sync_ws)) return MOE_ERR_ALIGNMENT;
  int nsm = 0;
  if ((s = sm_count(&nsm)) != MOE_OK) return s;
  cudaStream_t st = as_stream(stream);
  GemmPlan gu, sgu, dn, sdn;
  if ((s = plan_gate_up(sh_rows, H, sw, sh_a, nullptr, nullptr, sh_h_ws, nullptr, dev_status, &sgu)) != MOE_OK)
    return s;
  if ((s = plan_gate_up(rows, H, w, a, nullptr, offsets, h_ws, nullptr, dev_status, &gu)) != MOE_OK) return s;
  if ((s = plan_down(sh_rows, H, sw, sh_h_ws, nullptr, nullptr, nullptr, sh_out, dev_status, &sdn)) != MOE_OK)
    return s;
  if ((s = plan_down(rows, H, w, h_ws, nullptr, offsets, row_w, out, dev_status, &dn)) != MOE_OK) return s;
  FfnArgs f{};
  const GemmPlan* plans[4] = {&sgu, &gu, &sdn, &dn};
  for (int i = 0; i < 4; ++i) {
    f.tmA[i] = plans[i]->tmA;
    f.tmB[i] = plans[i]->tmB;
    f.g[i] = plans[i]->g;
  }
  f.ready = static_cast<int32_t*>(sync_ws);
  f.tile_counter = f.ready + nctr;
  f.shared_base = ffn_routed_blocks(rows, w->groups);
  cudaError_t e = cudaMemsetAsync(sync_ws, 0, need, st);
  if (e != cudaSuccess) return cuda_fail(e);
  return check_launch(launch_ffn_bf16(f, nsm, st));
}

moe_status moe_down_proj_combine(int32_t rows, int32_t T, int32_t H, const moe_ffn_weights* w, const void* h,
                                 const int32_t* offsets, const float* row_w, const int32_t* src_token,
                                 const moe_ffn_weights* sw, const void* sh_h, float* acc_ws, void* y,
                                 int32_t* dev_status, void* stream) {
  moe_status s = check_ffn(rows, H, w, h, nullptr, false, true);
  if (s != MOE_OK) return s;
  if (w->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (T < 1 || !offsets || !row_w || !src_token || !acc_ws || !y) return MOE_ERR_INVALID_ARG;
  if (sw) {
    if ((s = check_ffn(T, H, sw, sh_h, nullptr, false, true)) != MOE_OK) return s;
    if (sw->groups != 1 || sw->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  }
  if (any_misaligned(offsets, row_w, src_token, acc_ws, y)) return MOE_ERR_ALIGNMENT;
  int nsm = 0;
  if ((s = sm_count(&nsm)) != MOE_OK) return s;
  cudaStream_t st = as_stream(stream);
  cudaError_t e = cudaMemsetAsync(acc_ws, 0, static_cast<size_t>(T) * H * sizeof(float), st);
  if (e != cudaSuccess) return cuda_fail(e);
  GemmPlan p, q;
  if ((s = plan_down(rows, H, w, h, nullptr, offsets, row_w, acc_ws, dev_status, &p)) != MOE_OK) return s;
  p.g.scatter_tok = src_token;
  p.g.scatter_T = T;
  if (sw) {
    if ((s = plan_down(T, H, sw, sh_h, nullptr, nullptr, nullptr, acc_ws, dev_status, &q)) != MOE_OK) return s;
    q.g.scatter_tok = nullptr;
    q.g.scatter_T = T;
  }
  if ((s = launch_plan(p, EPI_SCATTER, st, nsm, sw ? &q : nullptr)) != MOE_OK) return s;
  return check_launch(launch_cast_rows(T, H, acc_ws, y, st));
}

moe_status moe_combine(int32_t T, int32_t k, int32_t H, const void* expert_out, const int32_t* slot_to_row,
                       const float* topk_w, const void* shared_out, void* y, void* stream) {
  if (T < 1 || k < 1 || H < 1 || !expert_out || !slot_to_row || !y) return MOE_ERR_INVALID_ARG;
  if (k > 16 || H % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(expert_out, slot_to_row, topk_w, shared_out, y)) return MOE_ERR_ALIGNMENT;
  return check_launch(launch_combine(T, k, H, expert_out, slot_to_row, topk_w, shared_out, y, as_stream(stream)));
}

moe_status moe_bias_update(int32_t E, int32_t T, int32_t k, const int32_t* expert_counts, float* bias,
                           float gamma, float* load_cv, void* stream) {
  if (E < 1 || T < 1 || k < 1 || !expert_counts || !bias) return MOE_ERR_INVALID_ARG;
  if (E > 1024) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(expert_counts, bias, load_cv)) return MOE_ERR_ALIGNMENT;
  return check_launch(launch_bias_update(E, T, k, expert_counts, bias, gamma, load_cv, as_stream(stream)));
}

moe_status moe_aux_loss_workspace_size(int32_t T, int32_t E, int32_t seq_len, size_t* bytes) {
  if (!bytes || T < 1 || E < 1 || seq_len < 1 || T % seq_len != 0) return MOE_ERR_INVALID_ARG;
  *bytes = aux_loss_workspace_bytes(T, E, seq_len);
  return MOE_OK;
}

moe_status moe_aux_loss(int32_t T, int32_t E, int32_t k, int32_t seq_len, int32_t scoring, const float* logits,
                        const int32_t* topk_ids, float alpha, float* aux_out, void* workspace,
                        size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (T < 1 || E < 1 || k < 1 || k > E || seq_len < 1 || T % seq_len != 0) return MOE_ERR_INVALID_ARG;
  if (scoring != MOE_SOFTMAX && scoring != MOE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (!logits || !topk_ids || !aux_out || !workspace) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < aux_loss_workspace_bytes(T, E, seq_len)) return MOE_ERR_INVALID_ARG;
  if (E > 256) return MOE_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(workspace) % 8 != 0 || reinterpret_cast<uintptr_t>(logits) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(topk_ids) % 4 != 0 || reinterpret_cast<uintptr_t>(aux_out) % 4 != 0)
    return MOE_ERR_ALIGNMENT;
  return check_launch(launch_aux_loss(T, E, k, seq_len, scoring, logits, topk_ids, alpha, aux_out, workspace,
                                      dev_status, as_stream(stream)));
}

moe_status moe_quantize_blocks(int32_t batch, int32_t N, int32_t K, const void* w, void* q, float* scale,
                               void* stream) {
  if (batch < 1 || N < 1 || K < 1 || !w || !q || !scale) return MOE_ERR_INVALID_ARG;
  if (N % 128 != 0 || K % 128 != 0 || batch > 65535 || N / 128 > 65535) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(w, q, scale)) return MOE_ERR_ALIGNMENT;
  return check_launch(launch_quant_blocks(batch, N, K, w, q, scale, as_stream(stream)));
}

moe_status moe_quantize_rows(int32_t M, int32_t K, const void* a, void* q, float* scale, void* stream) {
  if (M < 1 || K < 1 || !a || !q || !scale) return MOE_ERR_INVALID_ARG;
  if (K % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(a, q, scale)) return MOE_ERR_ALIGNMENT;
  return check_launch(launch_quant_rows(M, K, a, q, scale, as_stream(stream)));
}

moe_status moe_read_device_status(const int32_t* dev_status, int32_t* out, void* stream) {
  if (!dev_status || !out) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = as_stream(stream);
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, dev_status, sizeof(v), cudaMemcpyDeviceToHost, st);
  if (e != cudaSuccess) return cuda_fail(e);
  e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e);
  *out = v;
  if (v == 0) return MOE_OK;
  if (v == MOE_DEVSTAT_TIMEOUT) return MOE_ERR_DEVICE_TIMEOUT;
  return MOE_ERR_DEVICE_CHECK;
}

}  // extern "C"

namespace {

// [outer, inner] matrix stored through boxes of box_rows rows x 128 bytes,
// bf16 or fp32.
moe_status make_out_tmap(CUtensorMap* m, const void* ptr, bool f32, uint64_t inner, uint64_t outer, uint32_t box_rows) {
  const uint64_t esize = f32 ? 4 : 2;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * esize};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / esize), box_rows};
  return encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, dims, strides, box);
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Parts of moe_swiglu_ffn_backward's workspace.
struct BackwardWs {
  size_t d_gu, hw, partial, total;
};
BackwardWs backward_ws(int32_t rows, int32_t I) {
  BackwardWs b;
  const size_t r = static_cast<size_t>(rows);
  b.d_gu = 0;
  b.hw = align256(r * 2 * I * 2);
  b.partial = b.hw + align256(r * I * 2);
  b.total = b.partial + align256(r * (I / 32) * 4);
  return b;
}

// One weight-gradient product: C[g] [M, N] from A [rows, M] and B [rows, N].
moe_status plan_wgrad(WgradProblem* p, int32_t rows, int32_t groups, const void* A, int32_t M, const void* B, int32_t N,
                      void* out, bool f32) {
  p->a_flat = M % 64 != 0;
  moe_status s = p->a_flat ? make_tmap(&p->tmA, A, false, M, rows, 64) : make_block_tmap(&p->tmA, A, M, rows);
  if (s != MOE_OK) return s;
  if ((s = make_block_tmap(&p->tmB, B, N, rows)) != MOE_OK) return s;
  if ((s = make_out_tmap(&p->tmOut, out, f32, N, static_cast<uint64_t>(groups) * M, 32)) != MOE_OK) return s;
  p->M = M;
  p->N = N;
  p->n_blocks = (N + 255) / 256;
  p->m_blocks = (M + 255) / 256;
  p->per_group = p->m_blocks * p->n_blocks;
  p->tiles = groups * p->per_group;
  return MOE_OK;
}

int tiles_in_int(long long tiles) { return tiles < (1 << 20) ? static_cast<int>(tiles) : 1 << 20; }

bool grad_args_ok(moe_dtype grad_dtype, int32_t accumulate) {
  if (grad_dtype != MOE_BF16 && grad_dtype != MOE_F32) return false;
  return accumulate == 0 || (accumulate == 1 && grad_dtype == MOE_F32);
}

}  // namespace

extern "C" {

moe_status moe_swiglu_ffn_backward_workspace_size(int32_t rows, int32_t I, size_t* bytes) {
  if (!bytes || rows < 1 || I < 1) return MOE_ERR_INVALID_ARG;
  if (I % 128 != 0) return MOE_ERR_UNSUPPORTED;
  *bytes = backward_ws(rows, I).total;
  return MOE_OK;
}

moe_status moe_swiglu_ffn_backward(int32_t rows, int32_t H, const moe_ffn_weights* w, const void* a, const void* gu,
                                   const void* d_out, const int32_t* offsets, const float* row_w, void* d_a,
                                   void* d_w13, void* d_w2, moe_dtype grad_dtype, int32_t accumulate, float* d_row_w,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  moe_status s = check_ffn(rows, H, w, d_out, nullptr, d_a != nullptr, true);
  if (s != MOE_OK) return s;
  if (w->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (!gu || !workspace || (d_w13 && !a) || (!offsets && w->groups != 1)) return MOE_ERR_INVALID_ARG;
  if (!d_a && !d_w13 && !d_w2 && !d_row_w) return MOE_ERR_INVALID_ARG;
  if (!grad_args_ok(grad_dtype, accumulate)) return MOE_ERR_INVALID_ARG;
  const BackwardWs ws = backward_ws(rows, w->I);
  if (workspace_bytes < ws.total) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(a, gu, d_out, offsets, row_w, d_a, d_w13, d_w2, d_row_w, workspace)) return MOE_ERR_ALIGNMENT;
  const int32_t I = w->I;
  const size_t r = static_cast<size_t>(rows), weight = static_cast<size_t>(w->groups) * I * H;   // values of w2
  const size_t esize = grad_dtype == MOE_F32 ? 4 : 2;
  // the products run beside one another: d_a in the place of a or d_out would be read after being written
  if (!outputs_apart({{d_a, r * H * 2}, {d_w13, weight * 2 * esize}, {d_w2, weight * esize}, {d_row_w, r * 4}, {workspace, ws.total}},
                     {{a, r * H * 2}, {gu, r * I * 4}, {d_out, r * H * 2}, {row_w, r * 4}, {w->w13, weight * 4}, {w->w2, weight * 2},
                      offsets_span(offsets, w->groups)}))
    return MOE_ERR_INVALID_ARG;
  // output tiles of the weight gradients are counted in int32
  if (static_cast<long long>(w->groups) * (2 * I / 128) * (H / 256) > 0x3fffffffLL) return MOE_ERR_UNSUPPORTED;
  int nsm = 0;
  if ((s = sm_count(&nsm)) != MOE_OK) return s;
  cudaStream_t st = as_stream(stream);
  char* base = static_cast<char*>(workspace);
  void* d_gu = base + ws.d_gu;
  void* hw = base + ws.hw;
  float* partial = reinterpret_cast<float*>(base + ws.partial);

  // dh0 = d_out w2 and the activation's backward: d_gu, row_w * h, partial sums of d_row_w
  CUtensorMap tmA;
  HalfMaps tmB;
  s = make_train_weight_tmap(&tmA, w->w2, TRAIN_HIDDEN, w->tiled, w->groups, H, I, 1);
  if (s != MOE_OK) return s;
  if ((s = make_half_tmaps(&tmB, d_out, H, rows, offsets)) != MOE_OK) return s;
  TrainGemmArgs g;
  g.rows = rows;
  g.K = H;
  g.M = I;
  g.groups = w->groups;
  g.offsets = offsets;
  g.tiled = w->tiled;
  g.gu = static_cast<__nv_bfloat16*>(const_cast<void*>(gu));   // read only
  g.row_w = row_w;
  g.d_gu = static_cast<__nv_bfloat16*>(d_gu);
  g.h = static_cast<__nv_bfloat16*>(hw);
  g.partial = partial;
  g.status = dev_status;
  g.wait_ns = wait_limit();
  if ((s = check_launch(launch_train_gemm(TRAIN_HIDDEN, 1, tmA, tmB, g, nsm, st))) != MOE_OK) return s;
  const bool weights = d_w13 || d_w2;
  int rows_tiles = 0;                                  // of the kernel the weight gradients run beside
  if (d_row_w && !weights) {                           // else with the weight gradients
    s = check_launch(launch_row_w_grad(rows, I / 32, partial, offsets, w->groups, d_row_w, st));
    if (s != MOE_OK) return s;
  }
  if (d_a) {                                           // d_a = d_gu w13
    const int subs = train_subs(rows, w->groups, 2 * I, H, nsm);
    s = make_train_weight_tmap(&tmA, w->w13, TRAIN_ROWS, w->tiled, w->groups, 2 * I, H, subs);
    if (s != MOE_OK) return s;
    if ((s = make_half_tmaps(&tmB, d_gu, 2 * static_cast<uint64_t>(I), rows, offsets)) != MOE_OK) return s;
    g.K = 2 * I;
    g.M = H;
    g.out = static_cast<__nv_bfloat16*>(d_a);
    rows_tiles = tiles_in_int(train_tiles(rows, w->groups, H, subs * 256));
    if ((s = check_launch(launch_train_gemm(TRAIN_ROWS, subs, tmA, tmB, g, nsm, st))) != MOE_OK) return s;
  }
  if (weights) {
    WgradArgs q{};
    const bool f32 = grad_dtype == MOE_F32;
    if (d_w13) {
      s = plan_wgrad(&q.prob[q.n_prob++], rows, w->groups, d_gu, 2 * I, a, H, d_w13, f32);
      if (s != MOE_OK) return s;
    }
    if (d_w2) {
      s = plan_wgrad(&q.prob[q.n_prob++], rows, w->groups, d_out, H, hw, I, d_w2, f32);
      if (s != MOE_OK) return s;
    }
    q.rows = rows;
    q.groups = w->groups;
    q.offsets = offsets;
    q.f32 = f32;
    q.accumulate = accumulate;
    q.after = d_a ? 1 : 0;
    q.beside = rows_tiles;
    q.partial = partial;
    q.d_row_w = d_row_w;
    q.n_partial = I / 32;
    q.status = dev_status;
    q.wait_ns = wait_limit();
    s = check_launch(launch_wgrad(q, nsm, st));
  }
  return s;
}

moe_status moe_route_backward(int32_t T, int32_t E, int32_t k, moe_scoring scoring, int32_t norm_topk_prob,
                              float routed_scaling_factor, const float* logits, const int32_t* topk_ids,
                              const float* d_topk_w, const int32_t* slot_to_row, float* d_logits, void* d_logits_bf16,
                              int32_t* dev_status, void* stream) {
  if (T < 1 || E < 1 || k < 1 || k > E || !logits || !topk_ids || !d_topk_w || !d_logits) return MOE_ERR_INVALID_ARG;
  if (scoring != MOE_SOFTMAX && scoring != MOE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (k > 16 || E > 256 || E < 16 || E % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(T) * k > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(logits, topk_ids, d_topk_w, slot_to_row, d_logits, d_logits_bf16)) return MOE_ERR_ALIGNMENT;
  const size_t values = static_cast<size_t>(T) * E, slots = static_cast<size_t>(T) * k * 4;
  // a token's warp has read its logits before it writes: d_logits may take their place
  const Span in{d_logits != logits ? logits : nullptr, values * 4};
  if (!outputs_apart({{d_logits, values * 4}, {d_logits_bf16, values * 2}},
                     {in, {topk_ids, slots}, {d_topk_w, slots}, {slot_to_row, slots}}))
    return MOE_ERR_INVALID_ARG;
  return check_launch(launch_route_backward(T, E, k, scoring, norm_topk_prob ? 1 : 0, routed_scaling_factor, logits,
                                            topk_ids, d_topk_w, slot_to_row, d_logits, d_logits_bf16, dev_status,
                                            as_stream(stream)));
}

moe_status moe_gate_backward(int32_t T, int32_t H, int32_t E, const void* d_logits_bf16, const void* x,
                             const void* gate_w, const void* dx_in, void* dx, void* d_gate, moe_dtype grad_dtype,
                             int32_t accumulate, int32_t* dev_status, void* stream) {
  if (T < 1 || H < 1 || E < 1 || !d_logits_bf16 || (!dx && !d_gate)) return MOE_ERR_INVALID_ARG;
  if ((dx && !gate_w) || (d_gate && !x) || (dx_in && !dx)) return MOE_ERR_INVALID_ARG;
  if (!grad_args_ok(grad_dtype, accumulate)) return MOE_ERR_INVALID_ARG;
  if (H % 256 != 0 || E > 256 || E < 16 || E % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(d_logits_bf16, x, gate_w, dx_in, dx, d_gate)) return MOE_ERR_ALIGNMENT;
  const size_t rows_bytes = static_cast<size_t>(T) * H * 2, gate_values = static_cast<size_t>(E) * H;
  const Span in{dx_in != dx ? dx_in : nullptr, rows_bytes};          // dx_in may be dx, but not overlap it otherwise
  if (!outputs_apart({{dx, rows_bytes}, {d_gate, gate_values * (grad_dtype == MOE_F32 ? 4 : 2)}},
                     {{d_logits_bf16, static_cast<size_t>(T) * E * 2}, {x, rows_bytes}, {gate_w, gate_values * 2}, in}))
    return MOE_ERR_INVALID_ARG;
  int nsm = 0;
  moe_status s = sm_count(&nsm);
  if (s != MOE_OK) return s;
  cudaStream_t st = as_stream(stream);
  int rows_tiles = 0;
  if (dx) {                                            // dx = dx_in + d_logits gate
    CUtensorMap tmA;
    HalfMaps tmB;
    if ((s = make_train_weight_tmap(&tmA, gate_w, TRAIN_ROWS, 0, 1, E, H, 1)) != MOE_OK) return s;
    if ((s = make_half_tmaps(&tmB, d_logits_bf16, E, T, nullptr)) != MOE_OK) return s;
    TrainGemmArgs g;
    g.rows = T;
    g.K = E;
    g.M = H;
    g.out = static_cast<__nv_bfloat16*>(dx);
    g.add = static_cast<const __nv_bfloat16*>(dx_in);
    rows_tiles = tiles_in_int(train_tiles(T, 1, H, 256));
    g.status = dev_status;
    g.wait_ns = wait_limit();
    if ((s = check_launch(launch_train_gemm(TRAIN_ROWS, 1, tmA, tmB, g, nsm, st))) != MOE_OK) return s;
  }
  if (d_gate) {                                        // d_gate = d_logits^T x
    WgradArgs q{};
    if ((s = plan_wgrad(&q.prob[0], T, 1, d_logits_bf16, E, x, H, d_gate, grad_dtype == MOE_F32)) != MOE_OK) return s;
    q.n_prob = 1;
    q.rows = T;
    q.groups = 1;
    q.f32 = grad_dtype == MOE_F32;
    q.accumulate = accumulate;
    q.after = dx ? 1 : 0;
    q.beside = rows_tiles;
    q.status = dev_status;
    q.wait_ns = wait_limit();
    s = check_launch(launch_wgrad(q, nsm, st));
  }
  return s;
}

moe_status moe_quantize_mxfp4_rows(int32_t rows, int32_t K, const void* a, int32_t a_rows, const int32_t* src_rows, void* q,
                                   void* scale, int32_t* dev_status, void* stream) {
  if (rows < 1 || K < 1 || a_rows < 1 || !a || !q || !scale || (!src_rows && a_rows < rows)) return MOE_ERR_INVALID_ARG;
  if (K % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(a, src_rows, q, scale)) return MOE_ERR_ALIGNMENT;
  const size_t n = static_cast<size_t>(rows) * K;
  if (!outputs_apart({{q, n / 2}, {scale, n / 32}}, {{a, static_cast<size_t>(a_rows) * K * 2}, {src_rows, static_cast<size_t>(rows) * 4}}))
    return MOE_ERR_INVALID_ARG;
  return check_launch(launch_mx_quant_rows(rows, K, a, a_rows, src_rows, q, scale, dev_status, as_stream(stream)));
}

moe_status moe_dequantize_mxfp4_rows(int32_t rows, int32_t K, const void* q, const void* scale, void* out, void* stream) {
  if (rows < 1 || K < 1 || !q || !scale || !out) return MOE_ERR_INVALID_ARG;
  if (K % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(q, scale, out)) return MOE_ERR_ALIGNMENT;
  const size_t n = static_cast<size_t>(rows) * K;
  if (!outputs_apart({{out, n * 2}}, {{q, n / 2}, {scale, n / 32}})) return MOE_ERR_INVALID_ARG;
  return check_launch(launch_mx_dequant_rows(rows, K, q, scale, out, as_stream(stream)));
}

moe_status moe_quantize_mxfp4_weights(int32_t batch, int32_t N, int32_t K, const void* w, void* q, void* scale,
                                      void* stream) {
  if (batch < 1 || N < 1 || K < 1 || !w || !q || !scale) return MOE_ERR_INVALID_ARG;
  if (N % 128 != 0 || K % 128 != 0 || static_cast<long long>(batch) * N > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(w, q, scale)) return MOE_ERR_ALIGNMENT;
  const size_t n = static_cast<size_t>(batch) * N * K;
  if (!outputs_apart({{q, n / 2}, {scale, n / 32}}, {{w, n * 2}})) return MOE_ERR_INVALID_ARG;
  return check_launch(launch_mx_quant_weights(batch, N, K, w, q, scale, as_stream(stream)));
}

}  // extern "C"
