// Host-side declarations shared by the library's translation units:
// validated problem description, workspace layout and kernel launchers.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe_b200.h"

namespace moe {

// Tile sizes of the tensor-core grouped GEMMs (run by CTA pairs): a unit
// covers at most kTcBM token rows of one group (UMMA N) and kTcBN1 SwiGLU
// features (two pair UMMAs of M = 256: W1 rows and the same W3 rows) or
// kTcBN2 model columns of the down projection (two pair UMMAs of M = 256).
// With FP8 weights a unit covers at most kTcBM8 token rows: its bf16 weight
// tiles live in tensor memory beside the accumulators.
// The fp32 SIMT GEMMs use 64 x 64 tiles.
constexpr int kTcBM = 256;
constexpr int kTcBM8 = 160;
constexpr int kTcBN1 = 256;
constexpr int kTcBN2 = 512;
constexpr int kTcBNh = 256;  // backward, first GEMM: weight columns of its smaller units
constexpr int kSimtBM = 64;
constexpr int kSimtBN = 64;
constexpr int kChunkTokens = 32;  // dispatch: tokens per warp chunk
constexpr int kMaxRouted = 512;
constexpr int kMaxTopK = 16;
constexpr int kMaxDevices = 64;   // devices a process may use the library on

struct Problem {
  int64_t T;
  int d, F, N, ns, k, G, TG;
  int score_fn, normalize, group_score, dtype;
  float route_scale;
  int64_t R;          // routed rows = T * k
  int nsF;            // shared MLP width
  int elem;           // bytes per element of x / weights / y
};

// Byte offsets of every workspace region (all 256-byte aligned).
struct Layout {
  size_t status, sched, logits, idx, gates, chunk_counts, chunk_base, counts, offsets;
  size_t grp_row0, grp_rows, unit_base1, unit_base2, perm, slot_pos, gate_perm;
  size_t x_perm, h_perm, h_sh, y_rows, x_stage[2], y_stage[2];
  size_t total, total_host;
  size_t logits_bytes;
  int64_t n_chunks;
};

moe_status make_problem(const moe_cfg* cfg, int64_t T, Problem* p);
// `planes`: of partial logits; 0 for the router_k_splits(p) that a call of p.T tokens needs.
Layout make_layout(const Problem& p, int planes = 0);

struct DispatchBuffers {
  const int32_t* idx;
  int32_t* chunk_counts;
  int32_t* chunk_base;
  int32_t* counts;
  int32_t* offsets;
  int32_t* grp_row0;
  int32_t* grp_rows;
  int32_t* unit_base1;
  int32_t* unit_base2;
  int32_t* perm;
  int32_t* slot_pos;   // [T, k]: permuted rows of the token's experts, ascending expert
  float* gate_perm;
  const float* gates;
  unsigned* status;
};

// bf16 row-major [rows, cols] as a 2-D TMA tensor map with a box of
// box_cols x box_rows (128-byte swizzle and 256-byte L2 promotion when
// swizzle128, else dense). Elements outside the matrix load as zero; a null
// base or an empty matrix gives a zeroed map that must not be used.
bool make_tmap_bf16(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_cols,
                    uint32_t box_rows, bool swizzle128);
// uint8 row-major [rows, cols] (FP8 codes) with a box of box_cols bytes x
// box_rows rows, 256-byte L2 promotion, zero fill outside; swizzle_bytes 64
// gives the 64-byte swizzle (box_cols must then be 64), 0 none.
bool make_tmap_u8(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_cols,
                  uint32_t box_rows, int swizzle_bytes = 0);
// The same with a swizzle of 0, 64 or 128 bytes.
bool make_tmap_bf16_swz(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_cols,
                        uint32_t box_rows, int swizzle_bytes);

// bf16 (elem_bytes 2) or fp32 (4) tensor of rank 2 or 3, dims[0] contiguous,
// row_bytes[i] the stride of dims[i + 1] in bytes, with a 64- or 128-byte
// swizzled box; elements outside load as zero and are not stored. A null base
// or an empty tensor gives a zeroed map that must not be used.
bool make_tmap_nd(CUtensorMap* m, const void* base, int elem_bytes, int rank, const uint64_t* dims,
                  const uint64_t* row_bytes, const uint32_t* box, int swizzle_bytes, bool promote);

// Router: logits (FP32 pipes) then selection. The reduction over d is cut
// into S contiguous K ranges (S = `splits`, or router_k_splits(p) when
// splits is 0) whose partial logits land in S planes of [T, N] fp32 in
// `logits` (logits_bytes must cover them) and are added in a fixed order.
// A token's logits depend only on its own row, d and S, so every S gives
// deterministic bits and equal S gives equal bits at any T. `status` (may be
// null) receives MOE_DEV_* bits; logits_out [T, N] (may be null) the logits.
constexpr int kRouterTargetSms = 148;
constexpr int kMaxRouterSplits = 16;
constexpr int kRouterTileTokens = 64;  // tokens per CTA tile: S changes with T in steps of these
int router_k_splits(const Problem& p);
// Tokens from which S is 1, however many more there are.
int64_t router_unsplit_tokens(const Problem& p);
cudaError_t launch_router(const Problem& p, const void* x, const void* W_r, const float* b,
                          float* logits, size_t logits_bytes, int32_t* idx, float* gates,
                          unsigned* status, cudaStream_t s, int splits = 0, float* logits_out = nullptr);

// Histogram / scan / scatter; bm, bn1, bn2 select the GEMM tile grid that
// the unit tables describe.
cudaError_t launch_dispatch(const Problem& p, const DispatchBuffers& db, int bm, int bn1, int bn2,
                            cudaStream_t s);

// Tables of the grouped GEMMs straight from per-group row counts [p.N]
// (groups in order, rows contiguous): grp_row0, grp_rows and unit bases in db.
// Counts that are negative or do not sum to p.T set MOE_DEV_BAD_EXPERT and
// give empty groups; db.status and the kSchedCounters counters of `sched` (unit
// counters, and at kSchedReady the flag from dx to the weight gradients) are
// cleared first.
constexpr int kSchedReady = 2, kSchedCounters = 4;
cudaError_t launch_group_tables(const Problem& p, const int32_t* counts, const DispatchBuffers& db, int bm, int bn1,
                                int bn2, int* sched, cudaStream_t s);

// Expert-parallel row reorder between source-major and expert-major order
// of the blocks counts[W, E] (see ep_reorder_kernel).
cudaError_t launch_ep_reorder(const int32_t* counts, int W, int E, int64_t row_bytes, const void* src, void* dst,
                              bool to_expert_major, cudaStream_t s);

// x_perm[slot_pos[t, s]] = x[t] for every placed (token, slot) pair
// (status: the workspace's device status word, for the debug build's bounds checks)
cudaError_t launch_gather(const Problem& p, const void* x, const int32_t* slot_pos, void* x_perm,
                          unsigned* status, cudaStream_t s);

struct GemmArgs {
  const void* x;        // [T, d]
  const void* x_perm;   // [R, d]
  const void* W1;       // [N, F, d]
  const void* W3;
  const void* W2;       // [N, d, F]
  const void* Ws1;      // [nsF, d]
  const void* Ws3;
  const void* Ws2;      // [d, nsF]
  void* h_perm;         // [R, F]
  void* h_sh;           // [T, nsF]
  void* y_rows;         // [R + T, d]
  const int32_t* grp_row0;
  const int32_t* grp_rows;
  const int32_t* unit_base1;
  const int32_t* unit_base2;
  const float* gate_perm;
  unsigned* status;
  int* sched;           // [2] unit counters of the two tensor-core launches
  bool sched_clear = false;  // they are zero already
  // FP8 expert weights: W1 .. Ws2 above hold the e4m3 codes (uint8, same
  // shapes) and these their UE8M0 scales, one byte per 128 x 128 block
  bool fp8 = false;
  const uint8_t* W1s = nullptr;
  const uint8_t* W3s = nullptr;
  const uint8_t* W2s = nullptr;
  const uint8_t* Ws1s = nullptr;
  const uint8_t* Ws3s = nullptr;
  const uint8_t* Ws2s = nullptr;
  // training forward: the pre-activations [R, 2 F] (g, then u) are kept here
  void* gu = nullptr;
};

// Tensor-core (bf16) expert GEMMs: SwiGLU projection then gated down
// projection. `between` (optional) is recorded on s between the two
// launches; without it the down projection is launched with programmatic
// dependent launch and overlaps the SwiGLU GEMM's drain.
cudaError_t launch_expert_gemms_tc(const Problem& p, const GemmArgs& a, cudaStream_t s,
                                   cudaEvent_t between);
// fp32 SIMT expert GEMMs.
cudaError_t launch_expert_gemms_simt(const Problem& p, const GemmArgs& a, cudaStream_t s,
                                     cudaEvent_t between);

// Backward of the grouped experts (moe_experts_backward), after the unit
// tables of its row tiles are in place. gu [R, 2 F] as the forward kept it;
// dg, du, gh [R, F] and dgate_part [dgate_planes(p), R] are scratch: the
// gradients of g and u, gate * h, and partial sums of the gate gradient.
struct ExpertsBwdArgs {
  const void* x_rows;      // [R, d]
  const float* gate_rows;  // [R] or null (gate 1)
  const void* W1;          // [N, F, d]
  const void* W3;
  const void* W2;          // [N, d, F]
  const void* gu;
  const void* dy_rows;     // [R, d]
  void* dx_rows;           // [R, d] or null
  float* dgate_rows;       // [R] or null
  void* dW1;               // [N, F, d], or null (with dW3 and dW2)
  void* dW3;
  void* dW2;               // [N, d, F]
  int grad_dtype;          // of dW1, dW3, dW2
  bool accumulate;         // add to them (fp32 only)
  void* dg;
  void* du;
  void* gh;
  float* dgate_part;
  const int32_t* grp_row0;
  const int32_t* grp_rows;
  const int32_t* unit_base1;
  const int32_t* unit_base2;
  unsigned* status;
  int* sched;              // [kSchedCounters], zero
};
// Tensor-core sums over rows (the weight gradients, and the router's dx): for
// every group g and matrix i, out[g][m][n] = sum over the group's rows r of
// A[r][m] B[r][n], bf16 operands, fp32 accumulation.
struct WgradMatrix {
  const void* A;  // [rows, M], row stride lda elements (a multiple of 8)
  const void* B;  // [rows, N]
  void* out;      // [groups, M, N]
  int64_t M;
  int N;
  int64_t lda;
};
struct WgradArgs {
  WgradMatrix mat[3];
  int nmat, groups;
  int64_t rows;
  const int32_t* grp_row0;
  const int32_t* grp_rows;
  int grad_dtype;
  bool accumulate;   // fp32 only
  unsigned* status;
  // Null, or: the kernel before this one in the stream has itself waited for all
  // that this one reads, sets this flag then (see publish_waited()), and the two
  // write different buffers. This one need not wait for its end before its own work.
  const int* ready;
  int* publish;      // null, or the flag to set for such a kernel behind this one
  int max_pairs;     // CTA pairs to use at most (0: all)
  bool beside;       // an independent kernel follows that may run beside this one
};
// How the router's two bf16 products share the CTA pairs: the token ranges of dW_r
// (at most most_splits, whatever the tokens up to p.T), and the pairs of dx when it
// runs beside dW_r (0: before it).
struct RoutePlan {
  int splits, most_splits, dx_pairs;
};
RoutePlan plan_route_products(const Problem& p);
cudaError_t launch_wgrad_tc(const WgradArgs& a, cudaStream_t s);
int dgate_planes(const Problem& p);
int simt_train_tile(const Problem& p);  // fp32: rows of a tile of the training forward's products
int simt_bwd_tile(const Problem& p);    // and of the backward's row products
__host__ __device__ constexpr int simt_cols(int tile) { return tile < 32 ? 32 : tile; }  // and its columns
cudaError_t launch_experts_train_simt(const Problem& p, const GemmArgs& a, cudaStream_t s);
int dh_tile(const Problem& p);  // weight columns of a unit of the first GEMM: kTcBNh or kTcBN2
cudaError_t launch_experts_backward_tc(const Problem& p, const ExpertsBwdArgs& a, cudaStream_t s);
cudaError_t launch_experts_backward_simt(const Problem& p, const ExpertsBwdArgs& a, cudaStream_t s);
// dgate[r] = sum over the planes of part[plane][r], in a fixed order; nothing
// where *units, the number of units that wrote them, is zero.
cudaError_t launch_dgate_reduce(const float* part, int planes, int64_t rows, const int32_t* units, float* dgate,
                                cudaStream_t s);

// The gradient of the logits (see route_bwd.cu), and the row tables of the
// two products that follow: ints written to `tables` from the parameters.
constexpr int kMaxRouteSplits = 16;
enum RouteTable : int {
  kRtRow0 = 0,                               // [2] one group of T rows (fp32 products) ...
  kRtRows = 2,                               // [2]
  kRtUnits = 4,                              // [3] ... and its unit table
  kRtExperts = 7,                            // [1] N
  kRtSplit0 = 8,                             // [kMaxRouteSplits] token ranges of the split dW_r
  kRtSplitRows = kRtSplit0 + kMaxRouteSplits,
  kRtReady = kRtSplitRows + kMaxRouteSplits, // [1] 0: the flag between the two products
  kRouteTables
};
struct RouteDzArgs {
  const float* logits;      // [T, N]
  const int32_t* idx;       // [T, k]
  const float* dgates;      // [T, k], or by permuted row with slot_pos
  const int32_t* slot_pos;  // [T, k] or null
  int64_t T;
  int N, k, score_fn, normalize;
  float route_scale;
  unsigned* status;
  float* dz;                // [T, ld] fp32 (zero past N), or null:
  __nv_bfloat16* dz16;      // [T, ld]
  __nv_bfloat16* dz16_t;    // [N, ld_t], or null when not needed
  int64_t ld, ld_t;         // multiples of 8
  int32_t* tables;
  int32_t table_values[kRouteTables];
};
cudaError_t launch_route_dz(const RouteDzArgs& a, cudaStream_t s);
// dW [elems] = sum of n fp32 planes, in order (elems a multiple of 4).
cudaError_t launch_join_planes(const float* planes, int n, int64_t elems, void* dW, int grad_dtype, bool accumulate,
                               cudaStream_t s);

// The router's two backward products from dz.
struct RouteBwdArgs {
  const void* x;     // [T, d]
  const void* W_r;   // [N, d]
  void* dx;          // [T, d] or null
  void* dW_r;        // [N, d] or null
  int grad_dtype;
  bool accumulate;
  unsigned* status;
  const float* dz;   // as in RouteDzArgs
  const __nv_bfloat16* dz16;
  const __nv_bfloat16* dz16_t;
  int64_t ld, ld_t;
  int32_t* tables;
  int splits;        // token ranges of dW_r, summed from the planes when above 1
  float* planes;     // [splits, N, d] fp32
};
cudaError_t launch_route_products_tc(const Problem& p, const RouteBwdArgs& a, cudaStream_t s);
cudaError_t launch_route_products_simt(const Problem& p, const RouteBwdArgs& a, cudaStream_t s);

// Entry-point helpers shared by the ABI's translation units (moe_abi.cu).
moe_status make_group_problem(const moe_cfg* cfg, int64_t rows, Problem* p);
moe_status cuda_fail(cudaError_t e);
cudaError_t wait_host_outputs(const void* ws, cudaStream_t s);
cudaError_t note_device_use(const void* ws, cudaStream_t s);
inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// y[t] = sum over the token's rows slot_pos[t, 0..k) (ascending expert) of
// y_rows, plus the shared row y_rows[R + t]
cudaError_t launch_combine(const Problem& p, const void* y_rows, const int32_t* slot_pos, void* y,
                           cudaStream_t s);
// The same with the routed rows [R, d] and the shared rows [T, d] (or null) apart,
// and a second set of rows [T, d] added after them (or null).
cudaError_t launch_combine_rows(const Problem& p, const void* routed_rows, const void* shared_rows,
                                const int32_t* slot_pos, void* y, cudaStream_t s,
                                const void* more_rows = nullptr);

int device_sm_count();

// Launches a kernel with programmatic stream serialization: it may start while
// its predecessor in the stream ends, and orders itself with griddep_wait().
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t s,
                         const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Keeps e as this host thread's moe_last_cuda_error() value.
void record_cuda_error(cudaError_t e);

}  // namespace moe
