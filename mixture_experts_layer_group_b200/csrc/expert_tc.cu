// Grouped expert GEMMs on the 5th-generation tensor cores (tcgen05 + TMEM,
// operands staged by TMA), run by CTA pairs (clusters of 2) with pair UMMAs
// (cta_group::2) in "weights as M" orientation. Every pair MMA takes 256
// weight rows as its A operand (128 in each CTA's shared memory, M = 256)
// and the group's token rows as B (N = the tokens of the unit rounded up to
// 16, at most 256, half of them in each CTA), so each SM streams its own
// weight rows but only half of the token rows, and the MMA work follows the
// real number of tokens per expert instead of a padded row tile. A unit
// issues two pair MMAs (its two 128-row A halves per CTA) per K step on one
// shared token tile. Two launches per layer:
//
//   SwiGLU GEMM  unit = (group, 256 features, <= 256 tokens): CTA r holds
//                features 128 r .. 128 r + 127 of the unit; half 0 of its
//                rows is W1, half 1 the same rows of W3, so TMEM lane i holds
//                g and u of one feature for every token column; epilogue
//                h = silu(g) * u -> bf16
//                ("Routed expert:" / "Shared expert:" steps g = x W1,
//                u = x W3, a = g sigma(g), h = a (.) u)
//   gate GEMM    unit = (group, 512 model columns, <= 256 tokens):
//                E^T = W2 h^T; epilogue E * G (the token slot's gate; 1 for
//                the shared MLP) -> bf16 row of the slot
//                ("E_i = h W2", "y_routed = sum G_i E_i")
//
// The training modes (enum Mode) are the SwiGLU GEMM that also stores g and u,
// and the backward's products dh and dx, which take the weights transposed
// (MN-major tiles; see BwdParams). 57344 rows of 63 experts of 896 x 1280: SwiGLU
// 268 us, down 145, dh 228, dx 221; 8192 rows of 32 of 2048 x 7168: 492, 232, 289
// and 421 us (read of the weights alone 287, 143, 143 and 287 us).
//
// Groups 0..N-1 are the routed experts over their expert-contiguous token
// rows; group N is the fused shared MLP over all T tokens, in the same
// persistent launch. A group of more than 256 rows is cut into equal chunks.
// Units of one group are consecutive, weight-tile major and token-chunk
// minor. The pair's first CTA takes units from a global counter, so the
// chunks that share a weight tile start together (they read it once through
// L2) and the last units balance across SMs. The gate GEMM is launched with
// programmatic stream serialization and waits for the SwiGLU grid before its
// first load.
//
// CTA roles (320 threads, one CTA per SM, persistent; the same roles in both
// CTAs of a pair except the MMA issuer, which only the first CTA has):
//   warp 0      TMA producer (one elected lane). In CTA 0 it also takes unit ids and
//               hands them to both CTAs through shared-memory rings (the
//               peer's by an asynchronous store, see below). Stages
//               are variable-size pieces of a 208 KB byte ring: per 64-wide
//               K block, 32 KB of weights (two 128-row boxes) and one token
//               box of 32, 64 or 128 rows (4 / 8 / 16 KB; the TMA engine's
//               cost is per box); the bytes of both CTAs complete on CTA 0's
//               stage barrier; weights read by one unit only are evict-first
//   warp 1      TMEM owner (both CTAs, pair allocation) + UMMA issuer (CTA 0,
//               one elected lane): 2 x 4 pair MMAs (256 x N x 16) per stage. Each
//               CTA's TMEM holds two buffers of 2 x 128 fp32 columns: a unit
//               of <= 128 tokens takes one buffer (the next unit's MMAs
//               overlap its epilogue), a larger unit takes both (2 x 256)
//   warps 2..9  epilogue, two warps per TMEM lane quadrant taking turns on
//               32-token blocks: each warp reads its quadrant in the m16n8
//               layout (tcgen05.ld 16x256b), applies SwiGLU or the gate,
//               transposes the 32 x 32 block into its own 64-byte-swizzled
//               shared-memory tile with stmatrix.trans and writes it with one
//               TMA tensor store (a ragged last block with 64-byte row
//               stores); no barrier between epilogue warps per block
// With FP8 (e4m3) weights the same kernel runs 448 threads: the producer
// loads the codes (64-byte swizzled rows) and the token box into the ring,
// eight converter warps (one per TMEM lane quadrant and weight half)
// dequantise each stage's codes exactly into bf16 in tensor memory, and the
// pair MMAs read A from there and B from the ring (kind::f16 as above); four
// epilogue warps, one per quadrant.
// Every signal from one CTA of the pair to the other (a unit id, the
// release of a unit-ring slot or of an accumulator, an FP8 slot report) is
// an asynchronous store that completes transaction bytes on the receiving
// CTA's mbarrier (st.async), so no thread waits for a cross-CTA arrive; the
// MMA commits reach both CTAs' barriers by multicast.
// Every mbarrier wait is bounded; on a timeout a CTA records
// MOE_DEV_WAIT_TIMEOUT, drains its own copies and MMAs (bounded again),
// frees its tensor memory and exits.

#include <initializer_list>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kSlots = 8;                         // stages in flight at most
constexpr int kBK = 64;                           // bf16 per K chunk: one 128 B swizzle row
constexpr int kMaxTok = kTcBM;                    // tokens per unit (<= 256)
constexpr int kTokBox = 32;                       // token-row granule of a stage
constexpr int kBoxBytes = kTokBox * kBK * 2;      // 4 KB
constexpr int kTokMaps = 3;                       // token boxes of 32, 64 and 128 rows
constexpr int kHalfBytes = 128 * kBK * 2;         // 16 KB: 128 weight rows of one half
constexpr int kATileBytes = 2 * kHalfBytes;       // 32 KB: this CTA's rows of both halves
constexpr int kMaxTokBytes = (kMaxTok / 2 / kTokBox) * kBoxBytes;  // 16 KB: a CTA's largest token box
constexpr int kMaxStageBytes = kATileBytes + kMaxTokBytes;          // 48 KB
constexpr int kHalved = 512;                      // ring_ntok: the unit takes one weight half (tokens below it)
constexpr int kTmemCols = 512;                    // the pair allocation in each CTA
constexpr int kRing = 8;                          // unit ids in flight between the roles
constexpr int kTileBytes = 32 * 32 * 2;           // a warp's dense 32 x 32 bf16 tile (TMA store box)
constexpr int kA8Bytes = 2 * 128 * kBK;           // 16 KB: the fp8 codes of a CTA's 256 weight rows x 64 K
constexpr int kFp8Block = 128;                    // FP8 scale block (rows and columns)
constexpr int kASlots = 3;                        // FP8: dequantised weight stages in tensor memory
constexpr int kASlotCols = 2 * kBK / 2;           // FP8: columns of one slot (two halves x 64 bf16 / 2)

// Shared-memory and tensor-memory plan. bf16 weights: one ring of
// variable-size stages (this CTA's 256 weight rows x 64 K in bf16, then the
// token box), which the MMAs read in place; TMEM holds two accumulator
// buffers of 256 columns. FP8 weights: the ring holds the fp8 codes (16 KB,
// 64-byte swizzled rows) and the token box; the converter warps dequantise
// each stage's codes in registers into one of two weight slots in tensor
// memory (three slots, columns 320..511), from which the pair MMAs take A
// (B, the token box, stays in the ring); the accumulators share columns
// 0..319, so a unit covers at most 160 tokens.
//
// A wide plan (bf16 weights) gives every epilogue warp three transpose tiles
// instead of one, out of the ring: the training forward stores g, u and h of
// a block, the backward's first GEMM reads g and u and stores their gradients
// and gate * h.
template <bool FP8, bool WIDE = false>
struct Plan;
template <>
struct Plan<false, false> {
  static constexpr int kEpiWarps = 8;            // two per TMEM lane quadrant
  static constexpr int kCvtWarps = 4;            // (no converters; 4 keeps the arithmetic defined)
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kRingBytes = 52 * 4096;   // 208 KB
  static constexpr int kABytes = kATileBytes;    // weight bytes at the head of a stage
  static constexpr int kChunk = kTcBM;           // token rows of a unit at most
  static constexpr int kTokAlign = 16;           // MMA N granule
  static constexpr uint32_t kAccCols = 512;      // accumulator columns: two buffers of 256
  static constexpr int kBarrierBytes = 512;
  static constexpr int kTiles = 1;               // transpose tiles per epilogue warp
};
template <>
struct Plan<false, true> : Plan<false, false> {
  static constexpr int kRingBytes = 44 * 4096;   // 176 KB
  static constexpr int kTiles = 3;
};
template <>
struct Plan<true, false> {
  static constexpr int kEpiWarps = 4;            // one per TMEM lane quadrant
  static constexpr int kCvtWarps = 8;            // two per TMEM lane quadrant: one per weight half
  static constexpr int kThreads = 64 + 32 * (kEpiWarps + kCvtWarps);
  static constexpr int kRingBytes = 54 * 4096;   // 216 KB
  static constexpr int kABytes = kA8Bytes;
  static constexpr int kChunk = kTcBM8;
  static constexpr int kTokAlign = 32;           // N of an MMA with A in tensor memory
  static constexpr uint32_t kAccCols = 320;      // two buffers of 160; then the weight slots
  static constexpr int kBarrierBytes = 1024;
  static constexpr int kTiles = 1;
};
template <class PL>
__host__ __device__ constexpr int tile_bytes() {
  return PL::kEpiWarps * PL::kTiles * kTileBytes;
}
template <class PL>
constexpr int smem_bytes() {
  return PL::kRingBytes + tile_bytes<PL>() + 1024 + PL::kBarrierBytes;
}
static_assert(smem_bytes<Plan<false>>() <= 232448 && smem_bytes<Plan<true>>() <= 232448 &&
                  smem_bytes<Plan<false, true>>() <= 232448,
              "shared memory budget");
static_assert(kMaxStageBytes * 3 <= Plan<false, true>::kRingBytes, "ring holds three full stages");
static_assert((kA8Bytes + kMaxTokBytes) * 4 <= Plan<true>::kRingBytes, "FP8 ring holds four full stages");
static_assert(Plan<false>::kEpiWarps % 4 == 0 && Plan<true>::kEpiWarps % 4 == 0, "whole quadrants");
static_assert(Plan<true>::kCvtWarps == 8, "one converter warp per (TMEM lane quadrant, weight half)");
static_assert(2 * Plan<false>::kChunk <= (int)Plan<false>::kAccCols && 2 * Plan<true>::kChunk <= (int)Plan<true>::kAccCols &&
                  Plan<true>::kAccCols % 64 == 0 &&
                  Plan<true>::kAccCols + kASlots * kASlotCols <= (uint32_t)kTmemCols,
              "accumulators and weight slots fit the tensor memory");
static_assert(kMaxTok % (2 * kTokBox) == 0 && Plan<false>::kChunk <= kMaxTok && Plan<true>::kChunk <= kMaxTok &&
                  Plan<true>::kChunk % Plan<true>::kTokAlign == 0,
              "token chunk");

// The forward's two GEMMs, the SwiGLU GEMM that also keeps g and u, and the
// backward's two products on the weights (see BwdParams).
enum Mode : int { kSwiGLU = 0, kGateDown = 1, kSwiGLUKeep = 2, kDh = 3, kDx = 4, kDhWide = 5, kDownEdge = 6, kDxEdge = 7,
                  kKeepEdge = 8 };
__host__ __device__ constexpr bool is_keep(int mode) { return mode == kSwiGLUKeep || mode == kKeepEdge; }
__host__ __device__ constexpr bool is_down(int mode) { return mode == kGateDown || mode == kDownEdge; }
__host__ __device__ constexpr bool is_dx(int mode) { return mode == kDx || mode == kDxEdge; }
__host__ __device__ constexpr bool is_swiglu(int mode) { return mode == kSwiGLU || is_keep(mode); }
__host__ __device__ constexpr bool is_dh(int mode) { return mode == kDh || mode == kDhWide; }
__host__ __device__ constexpr bool is_bwd(int mode) { return is_dh(mode) || is_dx(mode); }
__host__ __device__ constexpr bool is_wide(int mode) { return is_keep(mode) || is_dh(mode); }
// One 128-row weight half per CTA instead of two: a unit then takes one of the
// two accumulator buffers whatever its tokens, and its epilogue overlaps the
// next unit's MMAs.
__host__ __device__ constexpr bool one_half(int mode) { return mode == kDh; }
// GEMMs of a matrix whose last unit has half its columns or fewer left
// (edge_halves()): that unit takes one half as well, 128 weight rows per CTA. The
// down and dx GEMMs have 256 columns of 512 then; the SwiGLU GEMM 128 features,
// whose half holds 64 rows of W1 over 64 rows of W3 in either CTA, and the
// warps of TMEM lanes 64 .. 127 hand u to those of lanes 0 .. 63 in shared memory.
// Modes of their own, because the decision per unit costs the other shapes 0.5 %.
__host__ __device__ constexpr bool may_halve(int mode) {
  return mode == kDownEdge || mode == kDxEdge || mode == kKeepEdge;
}
// Weight bytes at the head of a bf16 stage.
__host__ __device__ constexpr int a_bytes(int mode) { return one_half(mode) ? kHalfBytes : kATileBytes; }

struct TcParams {
  // bf16 weights: bf16 maps of 64 x 128 boxes (128-byte swizzle; the down
  // GEMM's A maps have 256-row boxes). FP8 weights: uint8 maps of the e4m3
  // codes, 64-byte x 128-row boxes (256 rows for the down GEMM), unswizzled.
  CUtensorMap a0_routed;  // W1 [N*F, d]      | W2 [N*d, F]
  CUtensorMap a1_routed;  // W3 [N*F, d]      | W2 in boxes of 128 rows (bf16)
  CUtensorMap a0_shared;  // Ws1 [nsF, d]     | Ws2 [d, nsF]
  CUtensorMap a1_shared;  // Ws3 [nsF, d]     | Ws2 in boxes of 128 rows (bf16)
  CUtensorMap b_routed[kTokMaps];  // x_perm [R, d] | h_perm [R, F]   (boxes of 32 / 64 / 128 rows)
  CUtensorMap b_shared[kTokMaps];  // x [T, d]      | h_sh [T, nsF]
  CUtensorMap o_routed;   // h_perm [R, F]    | y_rows [R + T, d]   (32 x 32 store box)
  CUtensorMap o_shared;   // h_sh [T, nsF]    | y_rows [R + T, d]
  const int32_t* unit_base;  // [N + 2]: units before group g; [N + 1] = total
  const int32_t* grp_row0;   // [N + 1]
  const int32_t* grp_rows;   // [N + 1]
  int* sched;                // unit counter, zero at launch
  int N;
  int k_routed, k_shared;        // reduction length (d | F, d | nsF)
  int cols_routed, cols_shared;  // output columns (F, nsF | d, d)
  int a_rows_per_expert;         // rows of the stacked weight tensor per routed expert (F | d)
  int tile_cols;                 // output columns per unit (256 | 512)
  __nv_bfloat16* out_routed;
  int64_t ld_routed;
  __nv_bfloat16* out_shared;
  int64_t ld_shared;
  int out_row0_shared;           // first row of the shared MLP's rows in o_shared (0 | R)
  const float* gate_perm;        // [R] (gate-down mode)
  unsigned* status;
  // FP8 weights: UE8M0 block scales [rows / 128, K / 128] of a0 / a1 (routed,
  // shared), and the number of 128-row blocks of each (for clamping)
  const uint8_t* s0_routed;
  const uint8_t* s1_routed;
  const uint8_t* s0_shared;
  const uint8_t* s1_shared;
  int sblocks_routed, sblocks_shared;
  int chunk_rows;                // token rows of a unit at most (Plan::kChunk)
  // rows of the token operand, weight and output tensors (routed | shared
  // group), for the debug build's bounds checks
  int64_t tok_rows_routed, tok_rows_shared;
  int64_t a_rows_routed, a_rows_shared;
  int64_t out_rows_routed, out_rows_shared;
};

// The training modes' further parameters.
//   kSwiGLUKeep  o_g, o_u: g and u halves of gu [R, 2 F]
//   kDh  q^T = W2^T dy^T: A = W2 [N, d, F] taken MN-major (M = 256, or in
//        kDhWide 512, of the F features, K = d), B = dy; epilogue dg, du, gate h -> o_g, o_u,
//        o_routed and the partial gate gradients
//   kDx  dx^T = W1^T dg^T + W3^T du^T: A = W1 then W3 [N, F, d] MN-major
//        (M = 512 of the d columns), B = dg then du; K = F twice
// A is one 3-D map per weight tensor (columns, rows of one expert, expert),
// so a box past the expert's last row or column loads zeros.
struct BwdParams : TcParams {
  CUtensorMap b1[kTokMaps];  // du (kDx)
  CUtensorMap a0_edge, a1_edge;  // W1 and W3 in boxes of 64 rows (kKeepEdge)
  CUtensorMap o_g, o_u;
  __nv_bfloat16* out_g;      // row stride ld_g
  __nv_bfloat16* out_u;
  int64_t ld_g;
  const __nv_bfloat16* gu;   // [R, 2 F] (kDh)
  float* part;               // [ceil(F / 32), R] partial gate gradients, or null (kDh)
  int* publish;              // the flag of publish_waited(), or null (kDx)
  int beside;                // the next kernel runs beside this one (kDx)
};
template <int MODE>
struct ParamsOf {
  using type = TcParams;
};
template <>
struct ParamsOf<kSwiGLUKeep> {
  using type = BwdParams;
};
template <>
struct ParamsOf<kKeepEdge> {
  using type = BwdParams;
};
template <>
struct ParamsOf<kDh> {
  using type = BwdParams;
};
template <>
struct ParamsOf<kDhWide> {
  using type = BwdParams;
};
template <>
struct ParamsOf<kDx> {
  using type = BwdParams;
};
template <>
struct ParamsOf<kDxEdge> {
  using type = BwdParams;
};

struct Unit {
  int g;        // group (N = shared MLP)
  int f;        // output-column tile
  int tok0;     // first token row of the chunk within the group
  int ntok;     // tokens in the chunk (1..256)
  int nchunks;  // chunks of the group
};

MOE_DEV Unit decode_unit(const TcParams& p, int u) {
  int lo = 0, hi = p.N;  // largest g with unit_base[g] <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ld_after_wait(p.unit_base + mid) <= u) lo = mid;
    else hi = mid - 1;
  }
  const int local = u - ld_after_wait(p.unit_base + lo);
  const int rows = ld_after_wait(p.grp_rows + lo);
  // a group's rows split into nc chunks of (almost) equal size, so the
  // chunks that share a weight tile run at the same pace and keep reading
  // its lines from L2 together
  const int nc = (rows + p.chunk_rows - 1) / p.chunk_rows;
  const int cs = (rows + nc - 1) / nc;
  Unit un;
  un.g = lo;
  un.f = local / nc;
  un.tok0 = (local % nc) * cs;
  const int left = rows - un.tok0;
  un.ntok = left < cs ? left : cs;
  un.nchunks = nc;
  return un;
}

// Accumulator placement over kCols columns (identical in both CTAs), by the
// unit's MMA width n (its tokens rounded up to the N granule): a unit with
// n <= kHalf (kCols / 4 rounded down to 32 columns) takes one of two
// buffers, at 0 or kCols / 2 (its halves at base and base + kHalf), so the
// next unit's MMAs overlap its epilogue; a wider unit takes both (halves at
// 0 and kCols / 2). bf16 (512 columns): buffers for n <= 128; FP8 (320):
// n <= 64. The MMA issuer and every epilogue thread replay the same
// sequence, so they agree on every placement.
// With one half per unit (kOne) every unit takes one of the two buffers.
template <uint32_t kCols, bool kOne>
struct AccPlan {
  static constexpr uint32_t kHalf = kOne ? kCols / 2 : (kCols / 4) & ~31u;
  uint32_t next = 0;
  MOE_DEV void place(int n, uint32_t& mask, uint32_t& base, uint32_t& stride) const {
    if (n > (int)kHalf) {
      mask = 3u;
      base = 0;
      stride = kCols / 2;
    } else {
      mask = 1u << next;
      base = next * (kCols / 2);
      stride = kHalf;
    }
  }
  MOE_DEV void advance(int n) { next = n > (int)kHalf ? 0u : next ^ 1u; }
};
// MMA width (N) of a unit of ntok tokens.
template <bool FP8>
MOE_DEV int mma_n(int ntok) { return (ntok + Plan<FP8>::kTokAlign - 1) & ~(Plan<FP8>::kTokAlign - 1); }

struct Shared {
  uint64_t full[kSlots];       // CTA 0: stage bytes of both CTAs landed
  uint64_t empty[kSlots];      // both: the pair MMAs finished reading the stage
  uint64_t acc_full[2];        // both: accumulator buffer complete
  uint64_t acc_empty[2];       // CTA 0: both CTAs' epilogues released the buffer (CTA 0's epilogue
                               // warps arrive, CTA 1's complete 4 transaction bytes each)
  uint64_t ring_full[kRing];   // both: unit id published
  uint64_t ring_empty[kRing];  // CTA 0: every reader of the pair took the id (CTA 0's readers
                               // arrive, CTA 1's complete 4 transaction bytes each)
  uint64_t drained;            // both: all pair MMAs completed
  uint32_t slot_off[kSlots];   // byte offset of each stage in the ring
  int ring[kRing];
  int ring_nk[kRing];          // CTA 0, for the MMA issuer: the unit's K blocks and tokens (0: none left)
  int ring_ntok[kRing];
  int epi_unit[2];             // the epilogue leader's unit for the epilogue warps
  int epi_info[2][5];          // its decoded (g, f, tok0, ntok) and first output row
  uint32_t tmem_base;
  int abort_flag;
  uint32_t consumed;           // stage fills the MMA issuer observed complete
  uint32_t sink;               // CTA 0: target of CTA 1's signalling stores (never read)
};
static_assert(sizeof(Shared) <= 512, "barrier block");

// The FP8 path's extra state (after Shared, inside the barrier block).
struct SharedFp8 {
  uint64_t conv_full[kASlots];   // CTA 0: both CTAs' converters wrote the weight slot in TMEM (CTA 0's
                                 // converters arrive, CTA 1's complete 4 transaction bytes)
  uint64_t conv_empty[kASlots];  // both: the pair MMAs finished reading the slot
  int cvt_unit[2];             // the converter leader's unit for the converter warps
  int cvt_info[2][2];          // its (g, f)
  int cvt_ok;                  // the leader's waits for the current stage succeeded
  uint32_t seen;               // stage fills this CTA's converters observed complete
  uint32_t peer_word[kASlots];   // CTA 0: target of CTA 1's signalling stores (never read)
};
static_assert(512 + sizeof(SharedFp8) <= Plan<true>::kBarrierBytes, "FP8 barrier block");

// Barrier among the epilogue warps only (id 1; id 0 is __syncthreads).
template <int kWarps>
MOE_DEV void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }
// Barrier among the FP8 converter warps only (id 2).
template <int kWarps>
MOE_DEV void cvt_sync() { asm volatile("bar.sync 2, %0;" ::"n"(32 * kWarps) : "memory"); }
// The two epilogue warps that share the blocks of a SwiGLU unit of one half (ids 0..3).
MOE_DEV void edge_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(3 + id) : "memory"); }

// Two e4m3 codes (bytes i and i + 1 of w, i = 0 or 2) -> the bf16 pair of
// their values times 2^-120. For a code s eeee mmm the bf16 bit pattern
// s 0000 eeee mmm 0000 has exponent field e and mantissa m / 8, i.e. the
// value 2^(e - 127) (1 + m / 8) for e > 0 and the bf16 subnormal 2^-126 m / 8
// for e = 0 (e4m3: 2^(e - 7) (1 + m / 8) and 2^-6 m / 8), and zero stays zero.
// One byte permute spreads the two codes into 16-bit lanes with the sign
// replicated into each high byte; a shift and a mask place the fields.
template <int kSel>
MOE_DEV uint32_t e4m3x2_to_bf16x2_scaled(uint32_t w) {
  uint32_t t;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(t) : "r"(w), "n"(kSel));
  return (t << 4) & 0x87F087F0u;
}

MOE_DEV uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// bf16 pair (f, f) with f = 2^e, -126 <= e <= 127.
MOE_DEV uint32_t bf16x2_pow2(int e) {
  const uint32_t b = (uint32_t)(e + 127) << 7;
  return b | (b << 16);
}

// 16 e4m3 codes -> 16 bf16 values, each code value times 2^(sb - 127):
// the values times 2^-120, multiplied by 2^(sb - 7) in one or (for
// sb - 7 > 127) two exact steps (a power of two times a bf16 with 4
// significant bits, subnormal or not, lands on a normal bf16).
MOE_DEV void dequant16(const uint4 w, int sb, uint32_t (&o)[8]) {
  const int e = sb - 7;                     // exponent of the total factor (>= -7)
  const int e1 = e > 127 ? 127 : e;
  const uint32_t f1 = bf16x2_pow2(e1);
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // bytes [b0, sign b0, b1, sign b1] and [b2, sign b2, b3, sign b3]
    o[2 * i] = mul_bf16x2(e4m3x2_to_bf16x2_scaled<0x9180>(words[i]), f1);
    o[2 * i + 1] = mul_bf16x2(e4m3x2_to_bf16x2_scaled<0xB3A2>(words[i]), f1);
  }
  if (e > 127) {
    const uint32_t f2 = bf16x2_pow2(e - 127);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = mul_bf16x2(o[i], f2);
  }
}

MOE_DEV int load_volatile(const int* p) { return *reinterpret_cast<const volatile int*>(p); }

constexpr int kMnBox = 64 * kBK * 2;  // 8 KB: 64 weight columns x 64 k

// K blocks of a unit: one segment of `seg` blocks, or two (dg W1, then du W3).
template <int MODE>
MOE_DEV int k_blocks(int seg) { return is_dx(MODE) ? 2 * seg : seg; }

// Writes one 64-byte token-row segment (32 bf16 from the transpose tile),
// or the first ncols of it at a ragged right edge.
MOE_DEV void store_row32(__nv_bfloat16* dst, int ncols, const uint4 (&v)[4]) {
  if (ncols >= 32) {
    uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
    for (int c = 0; c < 4; ++c) d4[c] = v[c];
  } else {
    const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(v);
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (c < ncols) dst[c] = e[c];
  }
}

// Address of a lane's row for the transposing matrix moves between a 32 x 32
// block in the accumulator's m16n8 layout and its [token][feature] tile (64-byte
// swizzled): matrix m of (hf, rp) is column group r = 2 rp + m / 2 and feature
// octet e = m % 2 of the lane half hf.
MOE_DEV uint32_t tile_row_addr(uint32_t tile, int hf, int rp) {
  const int lane = threadIdx.x & 31, m = lane >> 3, k = lane & 7;
  const int t = 8 * (2 * rp + (m >> 1)) + k;  // token row this lane addresses
  const int c = 2 * hf + (m & 1);             // feature chunk
  return tile + t * 64 + ((c ^ ((t >> 1) & 3)) << 4);
}

// g and u of one block (32 tokens x 32 features) of gu, 16 bytes per load.
struct GuBlock {
  uint4 v[2][4];
  MOE_DEV void load(const __nv_bfloat16* gu, int cols, int64_t row, int left, int c0) {
    const int lane = threadIdx.x & 31, c = c0 + 8 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 8 * i + (lane >> 2);
      const bool in = t < left && c < cols;  // 8 columns are all in or all out
      const __nv_bfloat16* src = gu + (row + t) * 2 * cols + c;
      v[0][i] = in ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
      v[1][i] = in ? __ldg(reinterpret_cast<const uint4*>(src + cols)) : make_uint4(0, 0, 0, 0);
    }
  }
  MOE_DEV void put(uint32_t tiles) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 8 * i + (lane >> 2);
      const uint32_t at = tiles + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4);
      st_shared_v4(at, v[0][i]);
      st_shared_v4(at + kTileBytes, v[1][i]);
    }
  }
};

// Epilogue of a kDh unit for one warp: blocks of 32 tokens x the warp's 32
// features of each half, q from tensor memory, g and u from gu. Per element,
// with s = sigma(g), act = g s, h = act u, dh = gate q:
//   dgate += q h   du = dh act   dg = dh u (s + s (g - act))   gh = gate h
// in packed fp32 pairs (two tokens). This is what bounds the product with K = 1280
// (57344 rows of 63 experts of 896 features): the warps never wait for an
// accumulator, and a block takes one about 5500 cycles, four blocks of a unit's
// 28,000 (its MMAs are 10,200). Of a block, issuing the next one's loads of g and u
// takes 1800, the move from tensor memory and the gate 1100, the arithmetic 1300
// (64 special-function operations per thread are 1000 for the two warps of a
// scheduler), the stores 600. The next block's g and u load meanwhile; the tiles of the
// three results are written in place of g and u (one TMA store each), and the
// sum over the block's features of q h is folded over the lanes after them.
MOE_DEV void dh_epilogue(const BwdParams& p, const Unit& un, int64_t row_base, uint32_t t_q, uint32_t stride, int halves,
                         uint8_t* tiles, int c_first, int sub, int subs) {
  const int lane = threadIdx.x & 31, cols = p.cols_routed;
  const uint32_t tile = smem_u32(tiles);
  const int tok_blocks = (un.ntok + 31) / 32;
  const int per_half = (tok_blocks - sub + subs - 1) / subs;  // this warp's blocks of a half (0: none)
  // (features at or past the matrix's width belong to a tile that reaches past it)
  if (halves == 2 && c_first + 128 >= cols) halves = 1;
  const int blocks = c_first >= cols ? 0 : halves * per_half;
  if (blocks <= 0) return;
  auto c_of = [&](int b) { return c_first + (b >= per_half ? 128 : 0); };
  auto j_of = [&](int b) { return 32 * (sub + subs * (b >= per_half ? b - per_half : b)); };
  GuBlock gu;
  gu.load(p.gu, cols, row_base + j_of(0), un.ntok - j_of(0), c_first);
#pragma unroll 1
  for (int b = 0; b < blocks; ++b) {
    const int c0 = c_of(b), j0 = j_of(b);
    const uint32_t t_b = t_q + (b >= per_half ? stride : 0) + j0;
    uint32_t a[2][16];
    tmem_ld16x256b_x4(t_b, a[0]);
    tmem_ld16x256b_x4(t_b + (16u << 16), a[1]);
    const int tok = j0 + lane;
    float my_gate = 1.0f;
    if (p.gate_perm && tok < un.ntok && MOE_IN_BOUNDS(row_base + tok < p.tok_rows_routed, p.status))
      my_gate = __ldg(p.gate_perm + row_base + tok);
    if (lane == 0) bulk_wait_group_read<0>();  // the previous block's stores have read the tiles
    __syncwarp();
    gu.put(tile);
    __syncwarp();
    if (b + 1 < blocks) gu.load(p.gu, cols, row_base + j_of(b + 1), un.ntok - j_of(b + 1), c_of(b + 1));
    uint64_t dgate[4], gate[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tq = 8 * r + 2 * (lane & 3);
      gate[r] = f32x2(__shfl_sync(0xffffffffu, my_gate, tq), __shfl_sync(0xffffffffu, my_gate, tq + 1));
      dgate[r] = 0;  // (0.0f, 0.0f)
    }
    tmem_wait_ld();
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t pg[4][2], pu[4][2], ph[4][2];
#pragma unroll
      for (int rp = 0; rp < 2; ++rp) {
        const uint32_t at = tile_row_addr(tile, hf, rp);
        ldmatrix_x4_trans(at, pg[2 * rp][0], pg[2 * rp][1], pg[2 * rp + 1][0], pg[2 * rp + 1][1]);
        ldmatrix_x4_trans(at + kTileBytes, pu[2 * rp][0], pu[2 * rp][1], pu[2 * rp + 1][0], pu[2 * rp + 1][1]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // four independent pairs side by side: the chain through the
        // exponential and the reciprocal is long
        uint64_t g[4], sg[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) g[r] = bf16x2_to_f32x2(pg[r][e]);
        sigmoid_f32x2(g, sg);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int x = 4 * r + 2 * e;
          const uint64_t q = f32x2(__uint_as_float(a[hf][x]), __uint_as_float(a[hf][x + 1]));
          const uint64_t u = bf16x2_to_f32x2(pu[r][e]);
          const uint64_t act = mul_f32x2(g[r], sg[r]), h = mul_f32x2(act, u), dh = mul_f32x2(gate[r], q);
          dgate[r] = fma_f32x2(q, h, dgate[r]);
          const uint64_t rest = fma_f32x2(act, f32x2(-1.0f, -1.0f), g[r]);  // g - act
          pg[r][e] = f32x2_to_bf16x2(mul_f32x2(mul_f32x2(dh, u), fma_f32x2(sg[r], rest, sg[r])));
          pu[r][e] = f32x2_to_bf16x2(mul_f32x2(dh, act));
          ph[r][e] = f32x2_to_bf16x2(mul_f32x2(gate[r], h));
        }
      }
      __syncwarp();  // every lane has read this half's chunks
#pragma unroll
      for (int rp = 0; rp < 2; ++rp) {
        const uint32_t at = tile_row_addr(tile, hf, rp);
        stmatrix_x4_trans(at, pg[2 * rp][0], pg[2 * rp][1], pg[2 * rp + 1][0], pg[2 * rp + 1][1]);
        stmatrix_x4_trans(at + kTileBytes, pu[2 * rp][0], pu[2 * rp][1], pu[2 * rp + 1][0], pu[2 * rp + 1][1]);
        stmatrix_x4_trans(at + 2 * kTileBytes, ph[2 * rp][0], ph[2 * rp][1], ph[2 * rp + 1][0], ph[2 * rp + 1][1]);
      }
    }
    if (j0 + 32 <= un.ntok && c0 + 32 <= cols) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        (void)MOE_IN_BOUNDS(row_base + j0 + 32 <= p.out_rows_routed, p.status);
        const int row = (int)(row_base + j0);
        tma_store_2d(&p.o_g, tiles, c0, row);
        tma_store_2d(&p.o_u, tiles + kTileBytes, c0, row);
        tma_store_2d(&p.o_routed, tiles + 2 * kTileBytes, c0, row);
        bulk_commit_group();
      }
    } else {
      __syncwarp();
      const int64_t row = row_base + tok;
      if (tok < un.ntok && c0 < cols && MOE_IN_BOUNDS(row < p.out_rows_routed, p.status)) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          uint4 rowv[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            rowv[c] = ld_shared_v4(tile + i * kTileBytes + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
          store_row32((i == 0 ? p.out_g : i == 1 ? p.out_u : p.out_routed) + row * cols + c0, cols - c0, rowv);
        }
      }
    }
    if (p.part) {
      // fold the 8 partial sums of the 8 lanes that share lane % 4 (each holds
      // other features of the same tokens): after the exchanges lane 4 j + i
      // holds the block's sum for token 8 (j / 2) + 2 i + j % 2
      float v[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) split_f32x2(dgate[r], v[2 * r], v[2 * r + 1]);
#pragma unroll
      for (int w = 4; w >= 1; w >>= 1) {
        const bool upper = lane & (4 * w);
#pragma unroll
        for (int i = 0; i < w; ++i) {
          const float keep = upper ? v[i + w] : v[i], give = upper ? v[i] : v[i + w];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * w);
        }
      }
      const int j = lane >> 2, t = j0 + 8 * (j >> 1) + 2 * (lane & 3) + (j & 1);
      if (c0 < cols && t < un.ntok && MOE_IN_BOUNDS(row_base + t < p.tok_rows_routed, p.status))
        p.part[(int64_t)(c0 >> 5) * p.tok_rows_routed + row_base + t] = v[0];
    }
  }
}

template <int MODE, bool FP8>
__global__ void __launch_bounds__(Plan<FP8>::kThreads, 1)
    expert_gemm_tc_kernel(const __grid_constant__ typename ParamsOf<MODE>::type p) {
  using PL = Plan<FP8, is_wide(MODE)>;
  constexpr int kRingBytes = PL::kRingBytes;
  constexpr int kEpiWarps = PL::kEpiWarps, kCvtWarps = PL::kCvtWarps, kTBytes = tile_bytes<PL>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* tiles = reinterpret_cast<float*>(smem + kRingBytes);
  Shared& sh = *reinterpret_cast<Shared*>(reinterpret_cast<uint8_t*>(tiles) + kTBytes);
  SharedFp8& shf = *reinterpret_cast<SharedFp8*>(reinterpret_cast<uint8_t*>(&sh) + 512);

  const int warp = uniform_warp_id();
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: issues the pair MMAs and takes the units
  const bool first = rank == 0;
  // Weight rows of this CTA. SwiGLU: rows 128 r .. 128 r + 127 of the unit's
  // 256 features, taken from W1 (half 0) and from W3 (half 1). Down GEMM:
  // rows 256 r .. 256 r + 255 of the unit's 512 output columns, one
  // contiguous 256-row box whose first and second 128 rows are halves 0 and
  // 1; so TMEM lane l of half h in CTA r is output column 256 r + 128 h + l.
  // One half: rows 128 r .. 128 r + 127 of the unit's 256.
  constexpr int kABytes = FP8 ? PL::kABytes : a_bytes(MODE);
  const int rank_rows = (is_swiglu(MODE) || one_half(MODE) ? 128 : 256) * (int)rank;
  // Readers of each unit id in each CTA (producer or MMA issuer, epilogue
  // leader, FP8 converter leader). The pair's cross-CTA signals are
  // asynchronous stores that complete transaction bytes on the other CTA's
  // barrier (st.async): a blocking cluster-scope mbarrier arrive costs the
  // signalling thread about 1000 cycles.
  constexpr int kRingReaders = FP8 ? 3 : 2;
  const int half_cols = is_swiglu(MODE) ? 0 : 128;
  constexpr int kEdgeRows = is_swiglu(MODE) ? 64 : 128;  // a CTA's output columns of a unit that takes one half
  // whether a unit does
  auto halved = [&](int f, bool shared) {
    constexpr int kCols = is_swiglu(MODE) ? kTcBN1 : kTcBN2;
    return may_halve(MODE) && f * kCols + kCols / 2 >= (shared ? p.cols_shared : p.cols_routed);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.acc_full[b], 1);
      mbar_init(&sh.acc_empty[b], kEpiWarps);
    }
    for (int q = 0; q < kRing; ++q) {
      mbar_init(&sh.ring_full[q], 1);
      // CTA 0's readers: MMA issuer, epilogue leader (and FP8 converter leader)
      mbar_init(&sh.ring_empty[q], kRingReaders);
    }
    mbar_init(&sh.drained, 1);
    sh.abort_flag = 0;
    sh.consumed = 0;
    if (FP8) {
      for (int c = 0; c < kASlots; ++c) {
        mbar_init(&shf.conv_full[c], 1);
        mbar_init(&shf.conv_empty[c], 1);
      }
      shf.seen = 0;
    }
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.a0_routed);
    for (int m = 0; m < kTokMaps; ++m) tma_prefetch_desc(&p.b_routed[m]);
    if (is_swiglu(MODE) || is_dx(MODE)) tma_prefetch_desc(&p.a1_routed);
  }
  if (warp == 1) {
    tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // barriers and tensor memory of both CTAs are ready
  tc_fence_after();
  // (programmatic launch: what a predecessor wrote, and what grids before it wrote, the
  // unit tables among that, is read only after it has finished)
  griddep_wait();
  if constexpr (is_dx(MODE)) {
    if (threadIdx.x == 64) {  // (not the producer: the release takes about 1 us)
      if (p.publish && blockIdx.x == 0) publish_waited(p.publish);
      if (p.beside) griddep_launch_dependents();
    }
  }
  const int total_units = ld_after_wait(p.unit_base + p.N + 1);
  const uint32_t tmem_base = sh.tmem_base;
  volatile int* abort_flag = &sh.abort_flag;
  auto peer = [&](const void* local) { return map_to_rank(smem_u32(local), rank ^ 1u); };
  auto in_first = [&](const void* local) { return map_to_rank(smem_u32(local), 0u); };

  uint32_t fills = 0;  // producer: stage fills issued
  if (warp == 0) {
    // ------------------------------------------------- scheduler + producer --
    // (the whole warp runs the loop, one elected lane issues: see elect_one())
    {
      // a weight tile read by one unit only is streamed once: evict it first;
      // tiles shared by the chunks of a large group, and the token rows (read
      // by every feature tile of their group), are kept in L2 as long as possible
      const uint64_t pol_once = policy_evict_first();
      const uint64_t pol_last = policy_evict_last();
      // Ring allocation (identical in both CTAs, so stage offsets match).
      // Stages are placed back to back in fill order and freed in the same
      // order by the pair MMAs' commits, so the bytes in use form one circular
      // interval [offset of the oldest unfreed fill, head). A stage that does
      // not fit before the end restarts at 0.
      uint32_t head = 0, oldest = 0;
      auto acquire = [&](uint32_t j, uint32_t sz, uint32_t& pos) -> bool {
        for (;;) {
          const uint32_t inflight = j - oldest;
          bool fits = false;
          if (inflight == 0) {
            pos = head + sz <= (uint32_t)kRingBytes ? head : 0u;
            fits = true;
          } else if (inflight < (uint32_t)kSlots) {
            const uint32_t tail =
                __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(&sh.slot_off[oldest % kSlots]), 0);
            if (tail < head) {  // in use: [tail, head)
              if (head + sz <= (uint32_t)kRingBytes) {
                pos = head;
                fits = true;
              } else if (sz <= tail) {
                pos = 0;
                fits = true;
              }
            } else if (head + sz <= tail) {  // in use wraps: [tail, end) + [0, head)
              pos = head;
              fits = true;
            }
          }
          if (fits) return true;
          // wait for the oldest fill to be consumed
          if (!__all_sync(0xffffffffu, mbar_wait_cluster_bounded(&sh.empty[oldest % kSlots], (oldest / kSlots) & 1u,
                                                                 abort_flag)))
            return false;
          ++oldest;
        }
      };
      bool ok = true;
      for (int i = 0;; ++i) {
        const int q = i % kRing;
        int u = 0;
        if (first) {
          ok = __all_sync(0xffffffffu, mbar_wait_cluster_bounded(&sh.ring_empty[q], ((i / kRing) & 1) ^ 1, abort_flag));
          if (!ok) break;
          if (lane == 0) {
            u = atomicAdd(p.sched, 1);
            if (u >= total_units) u = -1;
            // the id itself is the 4 transaction bytes of the peer's ring_full
            st_async_u32(peer(&sh.ring[q]), (uint32_t)u, peer(&sh.ring_full[q]));
            sh.ring[q] = u;
          }
        } else {
          // this CTA's ring_full phase: one arrival (here) and the 4 bytes of CTA 0's store
          if (lane == 0) mbar_arrive_expect_tx(&sh.ring_full[q], 4);
          ok = __all_sync(0xffffffffu, mbar_wait_cluster_bounded(&sh.ring_full[q], (i / kRing) & 1, abort_flag));
          if (!ok) break;
          u = load_volatile(&sh.ring[q]);
          __syncwarp();
          if (lane == 0) st_async_u32(in_first(&sh.sink), 0u, in_first(&sh.ring_empty[q]));
        }
        u = __shfl_sync(0xffffffffu, u, 0);
        Unit un{};
        int K = 0, row0 = 0;
        if (u >= 0) {
          un = decode_unit(p, u);
          for (int* v : {&un.g, &un.f, &un.tok0, &un.ntok, &un.nchunks}) *v = __shfl_sync(0xffffffffu, *v, 0);
          K = un.g == p.N ? p.k_shared : p.k_routed;
          row0 = __shfl_sync(0xffffffffu, ld_after_wait(p.grp_row0 + un.g), 0);
        }
        const int seg = (K + kBK - 1) / kBK;  // K blocks of a segment
        const int nk = k_blocks<MODE>(seg);
        if (first && lane == 0) {
          sh.ring_nk[q] = nk;
          sh.ring_ntok[q] = u < 0 ? 0 : un.ntok | (halved(un.f, un.g == p.N) ? kHalved : 0);
          mbar_arrive(&sh.ring_full[q]);
        }
        if (u < 0) {
          // no units left for this CTA: the down GEMM may start on SMs as
          // they free up
          if (!is_down(MODE) && lane == 0) griddep_launch_dependents();
          break;
        }
        const bool shared = un.g == p.N;
        const int half_n = mma_n<FP8>(un.ntok) / 2;  // token rows per CTA
        // one token box per stage, the smallest of 32 / 64 / 128 rows that
        // covers this CTA's rows (the TMA engine's cost is per box, so a
        // single box beats several small ones even with rows to spare)
        const int tmap = half_n <= kTokBox ? 0 : (half_n <= 2 * kTokBox ? 1 : 2);
        const int nbox = 1 << tmap;  // in 32-row granules
        const bool half = halved(un.f, shared);
        const uint32_t a_len = half ? kHalfBytes : kABytes;
        const uint32_t tx = a_len + nbox * kBoxBytes;
        // weight row (backward: first column of the expert's matrix)
        const int rowA = (shared || is_bwd(MODE) ? 0 : un.g * p.a_rows_per_expert) + un.f * p.tile_cols +
                         (half ? kEdgeRows * (int)rank : rank_rows);
        const int rowB = row0 + un.tok0 + (int)rank * half_n;
        // the unit's rows lie inside the group and its tensors (TMA clips a
        // box that reaches past them, and the last column tile of a matrix
        // whose height is not a multiple of the tile may start past it)
        (void)MOE_IN_BOUNDS(un.ntok >= 1 && un.ntok <= p.chunk_rows && un.tok0 >= 0 &&
                                row0 + un.tok0 + un.ntok <=
                                    (shared ? p.tok_rows_shared : p.tok_rows_routed) &&
                                rowA >= 0 && rowA < (shared ? p.a_rows_shared : p.a_rows_routed) + p.tile_cols,
                            p.status);
        const CUtensorMap* ta1 = shared ? &p.a1_shared : &p.a1_routed;
        const CUtensorMap* ta0 = half && is_down(MODE) ? ta1 : shared ? &p.a0_shared : &p.a0_routed;
        const CUtensorMap* tb = shared ? &p.b_shared[tmap] : &p.b_routed[tmap];
        const uint64_t pol = un.nchunks == 1 ? pol_once : pol_last;
        for (int kc = 0; kc < nk; ++kc, ++fills) {
          const uint32_t s = fills % kSlots;
          uint32_t pos = 0;
          if (!acquire(fills, tx, pos)) {
            ok = false;
            break;
          }
          head = pos + tx;
          (void)MOE_IN_BOUNDS(pos + tx <= (uint32_t)kRingBytes, p.status);
          if (lane == 0) sh.slot_off[s] = pos;
          __syncwarp();
          if (elect_one()) {
            uint8_t* a_dst = smem + pos;
            uint8_t* b_dst = a_dst + a_len;
            const uint32_t full_bar = in_first(&sh.full[s]);
            if (FP8) {
              // every CTA's bytes complete on its own stage barrier, which its
              // converter warps wait on; the codes are 64 bytes per row
              mbar_arrive_expect_tx(&sh.full[s], tx);
              tma_load_2d_hint(a_dst, ta0, &sh.full[s], kc * kBK, rowA, pol);
              if (MODE == kSwiGLU) tma_load_2d_hint(a_dst + kA8Bytes / 2, ta1, &sh.full[s], kc * kBK, rowA, pol);
              tma_load_2d_hint(b_dst, tb, &sh.full[s], kc * kBK, rowB, pol_last);
            } else if (first) {
              mbar_arrive_expect_tx(&sh.full[s], 2 * tx);  // this CTA's bytes and the peer's
            }
            if constexpr (is_bwd(MODE)) {
              // 256 (128) weight columns x 64 k as four (two) 64 x 64 boxes (8 KB each, rows of 128 bytes per k)
              const bool second = is_dx(MODE) && kc >= seg;
              const int k0 = (second ? kc - seg : kc) * kBK;
              const CUtensorMap* ta = second ? &p.a1_routed : ta0;
#pragma unroll
              for (int c = 0; c < kABytes / kMnBox; ++c)
                if (c * kMnBox < (int)a_len)
                  tma_load_3d_pair(a_dst + c * kMnBox, ta, full_bar, rowA + 64 * c, k0, un.g, pol);
              tma_load_2d_pair(b_dst, second ? &p.b1[tmap] : tb, full_bar, k0, rowB, pol_last);
            } else if (MODE == kKeepEdge && half) {
              if constexpr (MODE == kKeepEdge) {
                tma_load_2d_pair(a_dst, &p.a0_edge, full_bar, kc * kBK, rowA, pol);
                tma_load_2d_pair(a_dst + kHalfBytes / 2, &p.a1_edge, full_bar, kc * kBK, rowA, pol);
              }
              tma_load_2d_pair(b_dst, tb, full_bar, kc * kBK, rowB, pol_last);
            } else if (!FP8) {
              tma_load_2d_pair(a_dst, ta0, full_bar, kc * kBK, rowA, pol);  // SwiGLU: 128 W1 rows; down: 256 rows
              if (is_swiglu(MODE)) tma_load_2d_pair(a_dst + kHalfBytes, ta1, full_bar, kc * kBK, rowA, pol);
              tma_load_2d_pair(b_dst, tb, full_bar, kc * kBK, rowB, pol_last);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer (CTA 0) --
    if (first) {
      // The whole warp runs the loop and one elected lane issues: the
      // instruction operands then stay in uniform registers (see elect_one()).
      // Issued from a branch on the lane index instead, four pair MMAs with
      // their wait and commit cost about 610 cycles of issue at any N; so,
      // 290, and at N = 256 all of it hides behind the MMAs' 512.
      uint32_t consumed = 0;
      uint32_t uses[2] = {0u, 0u};
      AccPlan<PL::kAccCols, one_half(MODE)> plan;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return (bool)__all_sync(0xffffffffu, mbar_wait_cluster_bounded(bar, parity, abort_flag));
      };
      for (int i = 0; ok; ++i) {
        const int q = i % kRing;
        if (!wait(&sh.ring_full[q], (i / kRing) & 1)) {
          ok = false;
          break;
        }
        // K blocks and tokens of the unit (0 tokens: no unit left)
        const int nk = __shfl_sync(0xffffffffu, load_volatile(&sh.ring_nk[q]), 0);
        const int tok_word = __shfl_sync(0xffffffffu, load_volatile(&sh.ring_ntok[q]), 0);
        const int ntok = tok_word & (kHalved - 1);
        const bool half = may_halve(MODE) && (tok_word & kHalved);
        if (elect_one()) mbar_arrive_expect_tx(&sh.ring_empty[q], 4 * kRingReaders);  // and CTA 1's readers' stores
        if (ntok == 0) break;
        const int n = mma_n<FP8>(ntok);
        const uint32_t idesc = idesc_bf16_f32(256, (uint32_t)n) | (is_bwd(MODE) ? kIdescAMn : 0u);
        uint32_t mask, base, stride;
        plan.place(n, mask, base, stride);
        (void)MOE_IN_BOUNDS(n <= p.chunk_rows + PL::kTokAlign && base + (one_half(MODE) ? 0 : stride) + n <= PL::kAccCols, p.status);
        plan.advance(n);
        for (int b = 0; b < 2 && ok; ++b)
          if ((mask >> b) & 1u) {
            ok = wait(&sh.acc_empty[b], (uses[b] & 1u) ^ 1u);
            ++uses[b];
          }
        if (!ok) break;
        tc_fence_after();
        const uint32_t d0 = tmem_base + base, d1 = tmem_base + base + stride;
        for (int kc = 0; kc < nk; ++kc) {
          const uint32_t s = consumed % kSlots, ph = (consumed / kSlots) & 1u;
          // FP8: the converted slot of this fill (both CTAs' converters have
          // observed its bytes land before they released it)
          const uint32_t c = FP8 ? consumed % kASlots : 0u;
          const bool landed = FP8 ? wait(&shf.conv_full[c], (consumed / kASlots) & 1u) : wait(&sh.full[s], ph);
          if (!landed) {
            ok = false;
            break;
          }
          ++consumed;
          tc_fence_after();
          const uint32_t off =
              __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(&sh.slot_off[s]), 0);
          const uint32_t stage_addr = smem_u32(smem) + off;
          const uint64_t bdesc = smem_desc_sw128(stage_addr + (half ? kHalfBytes : kABytes));  // the token box follows the weights
          if (elect_one()) {
            if (FP8) {
              // A: the converted slot in tensor memory, 8 columns per 16 K
              const uint32_t a_t = tmem_base + PL::kAccCols + c * kASlotCols;
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk) {
                umma_bf16_pair_ts(d0, a_t + kk * 8, bdesc + kk * 2, idesc, (kc | kk) != 0);
                umma_bf16_pair_ts(d1, a_t + kBK / 2 + kk * 8, bdesc + kk * 2, idesc, (kc | kk) != 0);
              }
            } else {
              // 16 K are 32 bytes of a K-major row, 16 rows of 128 bytes of an MN-major tile
              const uint64_t adesc = is_bwd(MODE) ? smem_desc_sw128_mn(stage_addr, kMnBox) : smem_desc_sw128(stage_addr);
              constexpr int kStep = is_bwd(MODE) ? 2048 >> 4 : 2, kHalf = kHalfBytes >> 4;
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk) {
                umma_bf16_pair(d0, adesc + kk * kStep, bdesc + kk * 2, idesc, (kc | kk) != 0);
                if (!one_half(MODE) && !half)
                  umma_bf16_pair(d1, adesc + kHalf + kk * kStep, bdesc + kk * 2, idesc, (kc | kk) != 0);
              }
            }
            umma_commit_pair_both(smem_u32(&sh.empty[s]));
            if (FP8) umma_commit_pair_both(smem_u32(&shf.conv_empty[c]));
          }
          __syncwarp();
        }
        if (ok && elect_one()) {
          for (int b = 0; b < 2; ++b)
            if ((mask >> b) & 1u) {
              umma_commit_pair_both(smem_u32(&sh.acc_full[b]));
            }
        }
        __syncwarp();
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
      }
      // all pair MMAs have completed once `drained` fires (in both CTAs)
      if (elect_one()) umma_commit_pair_both(smem_u32(&sh.drained));
      if (lane == 0) sh.consumed = consumed;
      __syncwarp();
    }
    if (lane == 0) {
      int no_abort = 0;  // wait for the MMAs even when unwinding
      if (!mbar_wait_cluster_bounded(&sh.drained, 0, &no_abort)) set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
    }
    __syncwarp();
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------ epilogue --
    const int q = warp & 3;                  // TMEM lane quadrant this warp may access
    const int ew = warp - 2;                 // epilogue warp: its transpose tile
    const int sub = ew >> 2;                 // which of the quadrant's warps
    __nv_bfloat16* tile =
        reinterpret_cast<__nv_bfloat16*>(reinterpret_cast<uint8_t*>(tiles) + ew * PL::kTiles * kTileBytes);
    const bool leader = threadIdx.x == 64;
    uint32_t uses[2] = {0u, 0u};
    AccPlan<PL::kAccCols, one_half(MODE)> plan;
    for (int i = 0;; ++i) {
      // the leader takes the next unit and waits for its accumulator(s); the
      // epilogue warps then agree on the outcome and all run the unit or all leave
      if (leader) {
        int u = -2;
        const int qr = i % kRing;
        if (mbar_wait_cluster_bounded(&sh.ring_full[qr], (i / kRing) & 1, abort_flag)) {
          u = load_volatile(&sh.ring[qr]);
          if (first) mbar_arrive(&sh.ring_empty[qr]);
          else st_async_u32(in_first(&sh.sink), 0u, in_first(&sh.ring_empty[qr]));
          if (u >= 0) {
            const Unit un = decode_unit(p, u);
            sh.epi_info[i & 1][0] = un.g;
            sh.epi_info[i & 1][1] = un.f;
            sh.epi_info[i & 1][2] = un.tok0;
            sh.epi_info[i & 1][3] = un.ntok;
            sh.epi_info[i & 1][4] = un.g == p.N ? un.tok0 : ld_after_wait(p.grp_row0 + un.g) + un.tok0;
            uint32_t mask, base, stride;
            plan.place(mma_n<FP8>(un.ntok), mask, base, stride);
            bool ok = true;
            for (int b = 0; b < 2 && ok; ++b)
              if ((mask >> b) & 1u) ok = mbar_wait_cluster_bounded(&sh.acc_full[b], uses[b] & 1u, abort_flag);
            if (!ok) u = -2;
          }
        }
        if (u == -2) {
          *abort_flag = 1;
          set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
        }
        sh.epi_unit[i & 1] = u;
      }
      epi_sync<kEpiWarps>();
      const int u = load_volatile(&sh.epi_unit[i & 1]);
      if (u < 0) break;
      Unit un;
      un.g = load_volatile(&sh.epi_info[i & 1][0]);
      un.f = load_volatile(&sh.epi_info[i & 1][1]);
      un.tok0 = load_volatile(&sh.epi_info[i & 1][2]);
      un.ntok = load_volatile(&sh.epi_info[i & 1][3]);
      uint32_t mask, base, stride;
      plan.place(mma_n<FP8>(un.ntok), mask, base, stride);
      plan.advance(mma_n<FP8>(un.ntok));
      uses[0] += mask & 1u;
      uses[1] += (mask >> 1) & 1u;
      tc_fence_after();
      const bool shared = un.g == p.N;
      const int64_t row_base = load_volatile(&sh.epi_info[i & 1][4]);
      __nv_bfloat16* out_base = shared ? p.out_shared : p.out_routed;
      const int64_t ld = shared ? p.ld_shared : p.ld_routed;
      const int cols = shared ? p.cols_shared : p.cols_routed;
      const uint32_t t_q = tmem_base + ((uint32_t)(q * 32) << 16) + base;
      const bool half = halved(un.f, shared);
      const int halves = is_dh(MODE) ? 0 : is_swiglu(MODE) || half ? 1 : 2;
      // this warp's first output column of the unit
      const int c_first = un.f * p.tile_cols + (half ? kEdgeRows * (int)rank : rank_rows) + 32 * q;
      if constexpr (is_dh(MODE))
        dh_epilogue(p, un, row_base, t_q, stride, one_half(MODE) || half ? 1 : 2, reinterpret_cast<uint8_t*>(tile),
                    c_first, sub, kEpiWarps / 4);
#pragma unroll 1
      for (int hh = 0; hh < halves; ++hh) {
        // its 32 output columns of this half
        const int c0 = c_first + half_cols * hh;
#pragma unroll 1
        for (int j0 = 32 * sub; j0 < un.ntok; j0 += 32 * (kEpiWarps / 4)) {
          const int tok = j0 + lane;
          const int64_t row = row_base + tok;
          // gate of this lane's token, spread to the lanes that hold it below
          float my_gate = 1.0f;
          if (is_down(MODE) && !shared && p.gate_perm && tok < un.ntok &&
              MOE_IN_BOUNDS(row < p.tok_rows_routed, p.status))
            my_gate = __ldg(p.gate_perm + row);
          // The block (32 features = this quadrant's TMEM lanes, x 32 tokens =
          // columns j0..j0+31) in the m16n8 layout: lane half hf and column
          // group r give this thread features 16 hf + 8 e + lane / 4 (e = 0, 1)
          // and tokens 8 r + 2 (lane % 4) + 0..1, packed as bf16 pairs.
          uint32_t pk[2][4][2];
          uint32_t pg[2][4][2], pu[2][4][2];  // is_keep: g and u
          const int tq = 2 * (lane & 3);
          const uint32_t tile_addr = smem_u32(tile);
          if (MODE == kKeepEdge && half && q >= 2) {
            // u of the features of quadrant q - 2, in the layout that its warp reads it
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
            float4* u_out = reinterpret_cast<float4*>(tile) + lane;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t b[16];
              tmem_ld16x256b_x4(t_q + ((uint32_t)(16 * hf) << 16) + j0, b);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 4; ++i)
                u_out[32 * (4 * hf + i)] = make_float4(__uint_as_float(b[4 * i]), __uint_as_float(b[4 * i + 1]),
                                                       __uint_as_float(b[4 * i + 2]), __uint_as_float(b[4 * i + 3]));
            }
            edge_sync(2 * sub + (q & 1));  // written
            edge_sync(2 * sub + (q & 1));  // read
            continue;
          }
          const bool from_peer = MODE == kKeepEdge && half;
          // (the warp of quadrant q + 2 with the same blocks is epilogue warp 4 sub + q)
          const float4* u_in = reinterpret_cast<const float4*>(reinterpret_cast<const uint8_t*>(tiles) +
                                                               (4 * sub + q) * PL::kTiles * kTileBytes) + lane;
          if (from_peer) edge_sync(2 * sub + (q & 1));
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t a[16];
            tmem_ld16x256b_x4(t_q + ((uint32_t)(16 * hf) << 16) + hh * stride + j0, a);
            if (is_swiglu(MODE)) {
              uint32_t b[16];
              if (from_peer) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float4 v = u_in[32 * (4 * hf + i)];
                  b[4 * i] = __float_as_uint(v.x);
                  b[4 * i + 1] = __float_as_uint(v.y);
                  b[4 * i + 2] = __float_as_uint(v.z);
                  b[4 * i + 3] = __float_as_uint(v.w);
                }
              } else {
                tmem_ld16x256b_x4(t_q + ((uint32_t)(16 * hf) << 16) + stride + j0, b);  // u of the same features
              }
              tmem_wait_ld();
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int x = 4 * r + 2 * e;
                  const float g0 = __uint_as_float(a[x]), g1 = __uint_as_float(a[x + 1]);
                  const float u0 = __uint_as_float(b[x]), u1 = __uint_as_float(b[x + 1]);
                  if (is_keep(MODE)) {
                    const uint64_t g[1] = {f32x2(g0, g1)}, u = f32x2(u0, u1);
                    uint64_t sg[1];
                    sigmoid_f32x2(g, sg);
                    pg[hf][r][e] = pack_bf16x2(g0, g1);
                    pu[hf][r][e] = pack_bf16x2(u0, u1);
                    pk[hf][r][e] = f32x2_to_bf16x2(mul_f32x2(mul_f32x2(g[0], sg[0]), u));
                  } else {
                    pk[hf][r][e] = pack_bf16x2(silu_tanh(g0) * u0, silu_tanh(g1) * u1);
                  }
                }
            } else {
              tmem_wait_ld();
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                float g0 = 1.0f, g1 = 1.0f;
                if (is_down(MODE)) {
                  g0 = __shfl_sync(0xffffffffu, my_gate, 8 * r + tq);
                  g1 = __shfl_sync(0xffffffffu, my_gate, 8 * r + tq + 1);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int x = 4 * r + 2 * e;
                  pk[hf][r][e] = pack_bf16x2(__uint_as_float(a[x]) * g0, __uint_as_float(a[x + 1]) * g1);
                }
              }
            }
          }
          if (from_peer) edge_sync(2 * sub + (q & 1));  // u has been read
          // Transpose into this warp's [32 tokens][32 features] tile, 64-byte
          // swizzled (16-byte chunk c of token row t sits at chunk c ^ ((t >> 1) & 3)),
          // with four transposing matrix stores.
          if (lane == 0) bulk_wait_group_read<0>();  // the previous block's store has read the tile
          __syncwarp();
          auto put = [&](int i, const uint32_t (&v)[2][4][2]) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int rp = 0; rp < 2; ++rp)
                stmatrix_x4_trans(tile_row_addr(tile_addr + i * kTileBytes, hf, rp), v[hf][2 * rp][0],
                                  v[hf][2 * rp][1], v[hf][2 * rp + 1][0], v[hf][2 * rp + 1][1]);
          };
          put(0, pk);
          if constexpr (is_wide(MODE)) {
            put(1, pg);
            put(2, pu);
          }
          const bool full_block = j0 + 32 <= un.ntok && c0 + 32 <= cols;
          if (full_block) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              (void)MOE_IN_BOUNDS(row_base + j0 < (shared ? p.out_rows_shared : p.out_rows_routed), p.status);
              tma_store_2d(shared ? &p.o_shared : &p.o_routed, tile, c0,
                           (int)(row_base + j0) + (shared ? p.out_row0_shared : 0));
              if constexpr (is_wide(MODE)) {
                tma_store_2d(&p.o_g, tile + kTileBytes / 2, c0, (int)(row_base + j0));
                tma_store_2d(&p.o_u, tile + kTileBytes, c0, (int)(row_base + j0));
              }
              bulk_commit_group();
            }
          } else {
            __syncwarp();
            auto store_row = [&](int i, __nv_bfloat16* base, int64_t row_len) {
              uint4 rowv[4];
#pragma unroll
              for (int c = 0; c < 4; ++c)
                rowv[c] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(tile) + i * kTileBytes +
                                                          lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
              // (columns at or past the matrix's width belong to a tile that
              // reaches past it: nothing to store)
              if (tok < un.ntok && c0 < cols &&
                  MOE_IN_BOUNDS(row < (shared ? p.out_rows_shared : p.out_rows_routed), p.status))
                store_row32(base + row * row_len + c0, cols - c0, rowv);
            };
            store_row(0, out_base, ld);
            if constexpr (is_wide(MODE)) {
              store_row(1, p.out_g, p.ld_g);
              store_row(2, p.out_u, p.ld_g);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        for (int b = 0; b < 2; ++b)
          if ((mask >> b) & 1u) {
            if (!first) st_async_u32(in_first(&sh.sink), 0u, in_first(&sh.acc_empty[b]));
            else if (ew == 0) mbar_arrive_expect_tx(&sh.acc_empty[b], 4 * kEpiWarps);  // and CTA 1's warps' stores
            else mbar_arrive(&sh.acc_empty[b]);
          }
      }
    }
  } else if (FP8) {
    // ----------------------------------------- FP8 converters (kCvtWarps) --
    // Warp cw writes weight half cw / 4 of the rows in its TMEM lane quadrant:
    // per fill, in the producer's order, it waits (through a leader) for this
    // CTA's bytes and for a free weight slot, then each thread dequantises its
    // row's 64 codes (the 64-byte-swizzled box row: chunk c at c ^ (row / 2 % 4))
    // exactly into 32 columns of bf16 pairs, stores them to its TMEM lane and
    // the leader tells the MMA issuer once every converter's stores are done.
    const int cw = warp - (2 + kEpiWarps);   // 0 .. kCvtWarps - 1
    const int q = warp & 3;                  // TMEM lane quadrant this warp may access
    const int hsel = cw >> 2;                // weight half
    const int row = hsel * 128 + 32 * q + lane;  // row of the stage's code tile
    const bool cleader = cw == 0 && lane == 0;
    uint32_t j = 0;  // fills converted
    bool alive = true;
    for (int i = 0; alive; ++i) {
      if (cleader) {
        int u = -2;
        const int qr = i % kRing;
        if (mbar_wait_cluster_bounded(&sh.ring_full[qr], (i / kRing) & 1, abort_flag)) {
          u = load_volatile(&sh.ring[qr]);
          if (first) mbar_arrive(&sh.ring_empty[qr]);
          else st_async_u32(in_first(&sh.sink), 0u, in_first(&sh.ring_empty[qr]));
          if (u >= 0) {
            const Unit un = decode_unit(p, u);
            shf.cvt_info[i & 1][0] = un.g;
            shf.cvt_info[i & 1][1] = un.f;
          }
        }
        if (u == -2) {
          *abort_flag = 1;
          set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
        }
        shf.cvt_unit[i & 1] = u;
      }
      cvt_sync<kCvtWarps>();
      if (load_volatile(&shf.cvt_unit[i & 1]) < 0) break;
      const int g = load_volatile(&shf.cvt_info[i & 1][0]);
      const int f = load_volatile(&shf.cvt_info[i & 1][1]);
      const bool shared = g == p.N;
      const int K = shared ? p.k_shared : p.k_routed;
      const int nk = K / kBK;                 // K is a multiple of 128 on this path
      const int nkb = K / kFp8Block;          // <= 64
      const int rowA = (shared ? 0 : g * p.a_rows_per_expert) + f * p.tile_cols + rank_rows;
      const int sblocks = shared ? p.sblocks_shared : p.sblocks_routed;
      // this warp's 128-row block: SwiGLU W1 (half 0) or W3 (half 1) rows of
      // the same block; down GEMM two consecutive W2 blocks (a block past the
      // matrix, whose rows load as zeros, takes the last block's scales)
      const int rb = min(rowA / kFp8Block + (MODE == kSwiGLU ? 0 : hsel), sblocks - 1);
      const uint8_t* sc = (MODE == kSwiGLU && hsel ? (shared ? p.s1_shared : p.s1_routed)
                                                   : (shared ? p.s0_shared : p.s0_routed)) +
                          (int64_t)rb * nkb;
      // lane l holds the scale bytes of K blocks l and l + 32
      const int sL = lane < nkb ? __ldg(sc + lane) : 0, sH = lane + 32 < nkb ? __ldg(sc + lane + 32) : 0;
      for (int kc = 0; kc < nk; ++kc, ++j) {
        const uint32_t s = j % kSlots, c = j % kASlots;
        if (cleader) {
          const bool ok = mbar_wait_bounded(&sh.full[s], (j / kSlots) & 1u, abort_flag) &&
                          mbar_wait_cluster_bounded(&shf.conv_empty[c], ((j / kASlots) & 1u) ^ 1u, abort_flag);
          if (ok) shf.seen = j + 1;
          else {
            *abort_flag = 1;
            set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
          }
          shf.cvt_ok = ok;
        }
        cvt_sync<kCvtWarps>();
        if (!load_volatile(&shf.cvt_ok)) {
          alive = false;
          break;
        }
        tc_fence_after();  // the MMAs that read this slot before have completed
        const int kb = kc >> 1;  // 64-wide K block -> 128-wide scale block
        const int sb = __shfl_sync(0xffffffffu, kb < 32 ? sL : sH, kb & 31);
        const uint32_t raw = smem_u32(smem) + *reinterpret_cast<volatile uint32_t*>(&sh.slot_off[s]);
        (void)MOE_IN_BOUNDS(*reinterpret_cast<volatile uint32_t*>(&sh.slot_off[s]) + kA8Bytes <= (uint32_t)kRingBytes,
                            p.status);
        const uint32_t src = raw + row * kBK;
        uint4 wv[4];
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) wv[c4] = ld_shared_v4(src + ((c4 ^ ((row >> 1) & 3)) << 4));
        uint32_t o[32];
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {
          uint32_t v[8];
          dequant16(wv[c4], sb, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[8 * c4 + e] = v[e];
        }
        tmem_st32(tmem_base + ((uint32_t)(32 * q) << 16) + PL::kAccCols + c * kASlotCols + hsel * (kBK / 2), o);
        tmem_wait_st();
        tc_fence_before();
        cvt_sync<kCvtWarps>();
        if (cleader) {
          // CTA 1 signals through an asynchronous store (a blocking
          // cluster-scope arrive costs about 1000 cycles per stage)
          if (first) mbar_arrive_expect_tx(&shf.conv_full[c], 4);
          else st_async_u32(in_first(&shf.peer_word[c]), j, in_first(&shf.conv_full[c]));
        }
      }
    }
  }

  if (warp >= 2 && warp < 2 + kEpiWarps && lane == 0) bulk_wait_group_all();  // epilogue stores complete
  __syncthreads();
  if (warp == 0 && lane == 0 && (first || FP8)) {
    // wait for any stage fill that was issued but never observed complete
    // (bf16: the bytes of both CTAs land on the first CTA's stage barrier;
    // FP8: every CTA's land on its own and its converters observe them)
    for (uint32_t j = FP8 ? shf.seen : sh.consumed; j < fills; ++j) {
      const uint32_t s = j % kSlots, ph = (j / kSlots) & 1u;
      int dummy = 0;
      if (!mbar_wait_cluster_bounded(&sh.full[s], ph, &dummy)) {
        set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
        break;
      }
    }
  }
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still touch its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// Token / weight operand: 64 columns x box_rows rows, 128-byte swizzle.
bool make_tmap(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  return make_tmap_bf16(m, base, rows, cols, kBK, box_rows, true);
}

// Token operand maps with boxes of 32, 64 and 128 rows.
bool make_token_tmaps(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols) {
  for (int i = 0; i < kTokMaps; ++i)
    if (!make_tmap(&m[i], base, rows, cols, (uint32_t)(kTokBox << i))) return false;
  return true;
}

// Destination of the epilogue's 32 x 32 tile stores (64-byte swizzled tile).
bool make_store_tmap(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols) {
  return make_tmap_bf16_swz(m, base, rows, cols, 32, 32, 64);
}

// The same for one half (g or u) of gu [rows, 2 cols].
bool make_half_tmap(CUtensorMap* m, const void* gu, int64_t rows, int cols, int half) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, stride[1] = {(uint64_t)cols * 4};
  const uint32_t box[2] = {32, 32};
  return make_tmap_nd(m, static_cast<const uint8_t*>(gu) + (int64_t)half * cols * 2, 2, 2, dims, stride, box, 64, false);
}

// A weight tensor [N, rows, cols] for the backward: boxes of 64 columns x 64
// rows of one expert.
bool make_weight_tmap(CUtensorMap* m, const void* base, uint64_t n, uint64_t rows, uint64_t cols) {
  const uint64_t dims[3] = {cols, rows, n}, stride[2] = {cols * 2, rows * cols * 2};
  const uint32_t box[3] = {64, (uint32_t)kBK, 1};
  return make_tmap_nd(m, base, 2, 3, dims, stride, box, 128, true);
}

// FP8 weight codes: 64 bytes x box_rows rows, 64-byte swizzle (each
// converter thread reads one row; a warp's 32 rows then cover all banks).
bool make_tmap_codes(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  return make_tmap_u8(m, base, rows, cols, kBK, box_rows, 64);
}

template <int MODE, bool FP8>
cudaError_t launch_one(const typename ParamsOf<MODE>::type& prm, int max_units, cudaStream_t s, bool programmatic) {
  // per device: the shared-memory opt-in done and the resident cluster count
  static std::mutex mu;
  static int max_clusters_of[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e0 = cudaGetDevice(&dev);
  if (e0 != cudaSuccess) return e0;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(Plan<FP8>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = (smem_bytes<Plan<FP8, is_wide(MODE)>>());
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (max_clusters_of[dev] == 0) {
      cudaError_t e = cudaFuncSetAttribute(expert_gemm_tc_kernel<MODE, FP8>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, (smem_bytes<Plan<FP8, is_wide(MODE)>>()));
      if (e != cudaSuccess) return e;
      cfg.gridDim = dim3(2 * (device_sm_count() / 2), 1, 1);
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, expert_gemm_tc_kernel<MODE, FP8>, &cfg);
      if (e != cudaSuccess) return e;
      max_clusters_of[dev] = n > 0 ? n : 1;
    }
    clusters = max_clusters_of[dev];
  }
  if (max_units < clusters) clusters = max_units > 0 ? max_units : 1;
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.numAttrs = programmatic ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, expert_gemm_tc_kernel<MODE, FP8>, prm);
}

// Whether the last unit of a matrix of this width takes one half. 57344 rows of
// 896 features, d 1280 (units of 512, 512 and 256 columns): the training forward
// 433 us without, 402 with; the backward 825 and 803 (the best of 40 calls each).
bool edge_halves(int cols, int tile) { return (cols + tile / 2 - 1) / (tile / 2) % 2 == 1; }

}  // namespace

cudaError_t launch_expert_gemms_tc(const Problem& p, const GemmArgs& a, cudaStream_t s,
                                   cudaEvent_t between) {
  const int sms = device_sm_count();
  if (!a.sched_clear) {
    const cudaError_t err0 = cudaMemsetAsync(a.sched, 0, 2 * sizeof(int), s);
    if (err0 != cudaSuccess) return err0;
  }
  const bool fp8 = a.fp8;
  const int cm = fp8 ? Plan<true>::kChunk : Plan<false>::kChunk;  // token rows of a unit at most
  const int64_t chunks_bound = (p.R + cm - 1) / cm + p.N + (p.ns > 0 ? (p.T + cm - 1) / cm : 0);

  // weight maps: bf16 tiles, or the FP8 codes (plus their block scales)
  auto wmap = [&](CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
    return fp8 ? make_tmap_codes(m, base, rows, cols, box_rows) : make_tmap(m, base, rows, cols, box_rows);
  };
  BwdParams gk{};  // the training forward's further stores
  TcParams& g1 = gk;
  bool ok = wmap(&g1.a0_routed, a.W1, (uint64_t)p.N * p.F, p.d, 128) &&
            wmap(&g1.a1_routed, a.W3, (uint64_t)p.N * p.F, p.d, 128) &&
            wmap(&g1.a0_shared, a.Ws1, (uint64_t)p.nsF, p.d, 128) &&
            wmap(&g1.a1_shared, a.Ws3, (uint64_t)p.nsF, p.d, 128) &&
            make_token_tmaps(g1.b_routed, a.x_perm, (uint64_t)p.R, p.d) &&
            make_token_tmaps(g1.b_shared, p.ns ? a.x : nullptr, (uint64_t)p.T, p.d) &&
            make_store_tmap(&g1.o_routed, a.h_perm, (uint64_t)p.R, p.F) &&
            make_store_tmap(&g1.o_shared, p.ns ? a.h_sh : nullptr, (uint64_t)p.T, p.nsF);
  if (!ok) return cudaErrorInvalidValue;
  g1.out_row0_shared = 0;
  g1.unit_base = a.unit_base1;
  g1.grp_row0 = a.grp_row0;
  g1.grp_rows = a.grp_rows;
  g1.sched = a.sched;
  g1.N = p.N;
  g1.k_routed = p.d;
  g1.k_shared = p.d;
  g1.cols_routed = p.F;
  g1.cols_shared = p.nsF;
  g1.a_rows_per_expert = p.F;
  g1.tile_cols = kTcBN1;
  g1.out_routed = (__nv_bfloat16*)a.h_perm;
  g1.ld_routed = p.F;
  g1.out_shared = (__nv_bfloat16*)a.h_sh;
  g1.ld_shared = p.nsF;
  g1.gate_perm = nullptr;
  g1.status = a.status;
  g1.s0_routed = a.W1s;
  g1.s1_routed = a.W3s;
  g1.s0_shared = a.Ws1s;
  g1.s1_shared = a.Ws3s;
  g1.sblocks_routed = (int)((int64_t)p.N * p.F / kFp8Block);
  g1.sblocks_shared = p.nsF / kFp8Block;
  g1.chunk_rows = cm;
  g1.tok_rows_routed = p.R;
  g1.tok_rows_shared = p.T;
  g1.a_rows_routed = (int64_t)p.N * p.F;
  g1.a_rows_shared = p.nsF;
  g1.out_rows_routed = p.R;
  g1.out_rows_shared = p.T;
  const int64_t max_cols1 = p.F > p.nsF ? p.F : p.nsF;
  const int64_t units1 = chunks_bound * ((max_cols1 + kTcBN1 - 1) / kTcBN1);
  const int grid1 = (int)(units1 < sms ? units1 : sms);
  cudaError_t err;
  if (a.gu) {
    if (!make_half_tmap(&gk.o_g, a.gu, p.R, p.F, 0) || !make_half_tmap(&gk.o_u, a.gu, p.R, p.F, 1))
      return cudaErrorInvalidValue;
    gk.out_g = (__nv_bfloat16*)a.gu;
    gk.out_u = gk.out_g + p.F;
    gk.ld_g = 2 * (int64_t)p.F;
    const bool edge = edge_halves(p.F, kTcBN1);
    if (edge && (!make_tmap(&gk.a0_edge, a.W1, (uint64_t)p.N * p.F, p.d, 64) ||
                 !make_tmap(&gk.a1_edge, a.W3, (uint64_t)p.N * p.F, p.d, 64)))
      return cudaErrorInvalidValue;
    err = edge ? launch_one<kKeepEdge, false>(gk, grid1, s, a.sched_clear)
               : launch_one<kSwiGLUKeep, false>(gk, grid1, s, a.sched_clear);
  } else {
    err = fp8 ? launch_one<kSwiGLU, true>(g1, grid1, s, false) : launch_one<kSwiGLU, false>(g1, grid1, s, a.sched_clear);
  }
  if (err == cudaSuccess && between) err = cudaEventRecord(between, s);
  if (err != cudaSuccess) return err;

  TcParams g2{};
  ok = wmap(&g2.a0_routed, a.W2, (uint64_t)p.N * p.d, p.F, 256) &&
       wmap(&g2.a0_shared, a.Ws2, (uint64_t)p.d, p.nsF, 256) &&
       (fp8 || (make_tmap(&g2.a1_routed, a.W2, (uint64_t)p.N * p.d, p.F, 128) &&
                make_tmap(&g2.a1_shared, a.Ws2, (uint64_t)p.d, p.nsF, 128))) &&
       make_token_tmaps(g2.b_routed, a.h_perm, (uint64_t)p.R, p.F) &&
       make_token_tmaps(g2.b_shared, p.ns ? a.h_sh : nullptr, (uint64_t)p.T, p.nsF) &&
       make_store_tmap(&g2.o_routed, a.y_rows, (uint64_t)(p.R + p.T), p.d) &&
       make_store_tmap(&g2.o_shared, a.y_rows, (uint64_t)(p.R + p.T), p.d);
  if (!ok) return cudaErrorInvalidValue;
  g2.out_row0_shared = (int)p.R;
  g2.unit_base = a.unit_base2;
  g2.grp_row0 = a.grp_row0;
  g2.grp_rows = a.grp_rows;
  g2.sched = a.sched + 1;
  g2.N = p.N;
  g2.k_routed = p.F;
  g2.k_shared = p.nsF;
  g2.cols_routed = p.d;
  g2.cols_shared = p.d;
  g2.a_rows_per_expert = p.d;
  g2.tile_cols = kTcBN2;
  g2.out_routed = (__nv_bfloat16*)a.y_rows;
  g2.ld_routed = p.d;
  g2.out_shared = (__nv_bfloat16*)a.y_rows + p.R * (int64_t)p.d;
  g2.ld_shared = p.d;
  g2.gate_perm = a.gate_perm;
  g2.status = a.status;
  g2.s0_routed = a.W2s;
  g2.s0_shared = a.Ws2s;
  g2.sblocks_routed = (int)((int64_t)p.N * p.d / kFp8Block);
  g2.sblocks_shared = p.d / kFp8Block;
  g2.chunk_rows = cm;
  g2.tok_rows_routed = p.R;
  g2.tok_rows_shared = p.T;
  g2.a_rows_routed = (int64_t)p.N * p.d;
  g2.a_rows_shared = p.d;
  g2.out_rows_routed = p.R;
  g2.out_rows_shared = p.T;
  const int64_t units2 = chunks_bound * ((p.d + kTcBN2 - 1) / kTcBN2);
  const int grid2 = (int)(units2 < sms ? units2 : sms);
  // the down GEMM overlaps the SwiGLU GEMM's drain unless an event must be
  // recorded between the two
  if (!fp8 && edge_halves(p.d, kTcBN2)) return launch_one<kDownEdge, false>(g2, grid2, s, !between);
  return fp8 ? launch_one<kGateDown, true>(g2, grid2, s, !between) : launch_one<kGateDown, false>(g2, grid2, s, !between);
}

// Units of 512 features load 3/4 of the operand bytes per product, units of 256
// hide their epilogue behind the next unit's products. The epilogue costs the
// same at any K = d: with K = 7168 the whole backward of 8192 rows of 32 experts of
// 2048 features takes 1478 us with the first and 1510 with the second, with K =
// 1280 that of 57344 rows of 63 experts of 896 features 840 and 799 us. With few
// units of 512 the smaller ones spread the weights over more SMs.
int dh_tile(const Problem& p) {
  const int64_t chunks = p.R / kTcBM + (p.N < p.R ? p.N : p.R);  // about one partly filled unit row per group
  return p.d > 2048 && chunks * ((p.F + kTcBN2 - 1) / kTcBN2) >= device_sm_count() / 4 ? kTcBN2 : kTcBNh;
}

int dgate_planes(const Problem& p) {
  const int cols = p.dtype == MOE_BF16 ? 32 : simt_cols(simt_bwd_tile(p));
  return (p.F + cols - 1) / cols;
}

cudaError_t launch_experts_backward_tc(const Problem& p, const ExpertsBwdArgs& a, cudaStream_t s) {
  const int sms = device_sm_count();
  constexpr int cm = Plan<false>::kChunk;
  const int64_t chunks_bound = (p.R + cm - 1) / cm + p.N;
  auto grid_of = [&](int cols, int tile) {
    const int64_t units = chunks_bound * ((cols + tile - 1) / tile);
    return (int)(units < sms ? units : sms);
  };

  BwdParams h{};
  bool ok = make_weight_tmap(&h.a0_routed, a.W2, p.N, p.d, p.F) && make_token_tmaps(h.b_routed, a.dy_rows, p.R, p.d) &&
            make_store_tmap(&h.o_routed, a.gh, p.R, p.F) && make_store_tmap(&h.o_g, a.dg, p.R, p.F) &&
            make_store_tmap(&h.o_u, a.du, p.R, p.F);
  if (!ok) return cudaErrorInvalidValue;
  h.unit_base = a.unit_base1;
  h.grp_row0 = a.grp_row0;
  h.grp_rows = a.grp_rows;
  h.sched = a.sched;
  h.N = p.N;
  h.k_routed = p.d;
  h.cols_routed = p.F;
  h.tile_cols = dh_tile(p);
  h.out_routed = (__nv_bfloat16*)a.gh;
  h.ld_routed = p.F;
  h.out_g = (__nv_bfloat16*)a.dg;
  h.out_u = (__nv_bfloat16*)a.du;
  h.ld_g = p.F;
  h.gate_perm = a.gate_rows;
  h.status = a.status;
  h.chunk_rows = cm;
  h.tok_rows_routed = h.out_rows_routed = p.R;
  h.a_rows_routed = p.F;
  h.gu = (const __nv_bfloat16*)a.gu;
  h.part = a.dgate_rows ? a.dgate_part : nullptr;
  cudaError_t err = dh_tile(p) == kTcBN2 ? launch_one<kDhWide, false>(h, grid_of(p.F, kTcBN2), s, true)
                                         : launch_one<kDh, false>(h, grid_of(p.F, kTcBNh), s, true);
  if (err != cudaSuccess) return err;

  // With few rows per group the dx GEMM is bound by reading the weights and the
  // weight gradients by writing them (a B200 writes 3.9 TB/s), and both need only
  // the dh GEMM: they then run beside each other, each on a part of the GPU. 32
  // experts of 2048 x 7168: 1073 instead of 1135 us with 128 rows each; with 256
  // there is nothing left to win (1497 against 1479). 16 experts of 896 x 1280
  // with 37 rows in all: 78 instead of 89 us.
  const int pairs = sms / 2;
  const bool beside = a.dx_rows && a.dW1 && p.R <= (int64_t)p.N * 192;
  const int dx_pairs = pairs * 3 / 7;
  if (a.dx_rows) {
    BwdParams x{};
    ok = make_weight_tmap(&x.a0_routed, a.W1, p.N, p.F, p.d) && make_weight_tmap(&x.a1_routed, a.W3, p.N, p.F, p.d) &&
         make_token_tmaps(x.b_routed, a.dg, p.R, p.F) && make_token_tmaps(x.b1, a.du, p.R, p.F) &&
         make_store_tmap(&x.o_routed, a.dx_rows, p.R, p.d);
    if (!ok) return cudaErrorInvalidValue;
    x.unit_base = a.unit_base2;
    x.grp_row0 = a.grp_row0;
    x.grp_rows = a.grp_rows;
    x.sched = a.sched + 1;
    x.N = p.N;
    x.k_routed = p.F;
    x.cols_routed = p.d;
    x.tile_cols = kTcBN2;
    x.out_routed = (__nv_bfloat16*)a.dx_rows;
    x.ld_routed = p.d;
    x.status = a.status;
    x.chunk_rows = cm;
    x.tok_rows_routed = x.out_rows_routed = p.R;
    x.a_rows_routed = p.d;
    x.publish = a.dW1 ? a.sched + kSchedReady : nullptr;
    x.beside = beside;
    const int grid = grid_of(p.d, kTcBN2);
    const int ctas = beside && grid > dx_pairs ? dx_pairs : grid;
    err = edge_halves(p.d, kTcBN2) ? launch_one<kDxEdge, false>(x, ctas, s, true) : launch_one<kDx, false>(x, ctas, s, true);
    if (err != cudaSuccess) return err;
  }
  // (last: between the GEMMs its launch and its wait would stand in their way)
  auto reduce_dgate = [&] {
    return a.dgate_rows ? launch_dgate_reduce(a.dgate_part, dgate_planes(p), p.R, a.unit_base1 + p.N + 1,
                                              a.dgate_rows, s)
                        : cudaSuccess;
  };
  if (!a.dW1) return reduce_dgate();
  WgradArgs w{};
  w.mat[0] = {a.dg, a.x_rows, a.dW1, p.F, p.d, p.F};
  w.mat[1] = {a.du, a.x_rows, a.dW3, p.F, p.d, p.F};
  w.mat[2] = {a.dy_rows, a.gh, a.dW2, p.d, p.F, p.d};
  w.nmat = 3;
  w.groups = p.N;
  w.rows = p.R;
  w.grp_row0 = a.grp_row0;
  w.grp_rows = a.grp_rows;
  w.grad_dtype = a.grad_dtype;
  w.accumulate = a.accumulate;
  w.status = a.status;
  w.ready = a.dx_rows ? a.sched + kSchedReady : nullptr;  // the dx GEMM has waited for the dh GEMM
  w.max_pairs = beside ? pairs - dx_pairs : 0;
  err = launch_wgrad_tc(w, s);
  return err == cudaSuccess ? reduce_dgate() : err;
}

}  // namespace moe
