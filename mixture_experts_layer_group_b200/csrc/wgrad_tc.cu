// Weight gradients on the tensor cores: dW[g][m][n] = sum over the rows r of
// group g of A[r][m] B[r][n], for several matrices in one launch (the
// experts' dW1 = dg^T x, dW3 = du^T x, dW2 = dy^T (gate h); the router's
// dW_r = dz^T x, and its dx = (dz^T)^T W_r over the experts as rows). Both operands are row-major with the rows as the reduction,
// so both are MN-major tiles: a 64 x 64 TMA box is 64 rows (k) of 128 bytes.
//
// CTA pairs (clusters of 2, cta_group::2): a unit is two 256 x 256 tiles of
// one group's matrix that share an operand (side by side along M or along N;
// one tile at an odd edge). Per 64 rows CTA r loads 128 columns of the shared
// operand and 128 of each tile's own (48 KB, four stages), and keeps rows 128 r
// .. 128 r + 127 of each tile in its tensor memory (256 columns a tile). What
// bounds a long sum is the operands' way from L2: 48 KB feed 1024 cycles of
// pair MMAs; with one tile per unit it was 64 KB, and the MMAs waited a quarter
// of their time. A unit of one tile takes one of the two buffers, so it overlaps
// its neighbour; between units of two tiles the first tile's MMAs of two stages
// run while the second tile is still being read. Units are taken with a fixed
// stride.
//
// A group's last stage may hold up to 15 rows of the next group inside its
// last K = 16 step. They would enter the sum, and a NaN there cannot be
// multiplied away, so a fixer warp in each CTA zeroes them in both operands
// before the stage is handed to the MMA issuer.
//
// Warps: 0 producer, 1 tensor-memory owner and MMA issuer (first CTA), 2..9
// epilogue (two per lane quadrant), 10 fixer. Waits are bounded as everywhere.
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kBK = 64;
constexpr int kTile = 256;
constexpr int kBox = 64 * kBK * 2;           // 8 KB
constexpr int kPart = 2 * kBox;              // 128 columns of an operand
constexpr int kStageBytes = 3 * kPart;       // the shared operand, then each tile's own
constexpr int kStages = 4;
constexpr int kLead = 2;                     // stages whose second tile follows later at a unit's start
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (3 + kEpiWarps);
constexpr int kOutTile = 32 * 128;           // 32 rows x 128 bytes per epilogue warp
constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kOutTile + 1024 + 512;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kTmemCols = 512;

struct Matrix {
  CUtensorMap a;    // [R, M]
  CUtensorMap b;    // [R, N]
  CUtensorMap out;  // [groups, M, N]
  int M, N, mt, nt;  // units along M and N
  int split_m;       // a unit's tiles lie along M (else along N)
  int per_unit;      // tiles of a unit at most: 1 or 2
};
struct Params {
  Matrix mat[3];
  int nmat, groups;
  int units_per_group, units;
  const int32_t* grp_row0;
  const int32_t* grp_rows;
  int accumulate;
  unsigned* status;
  int independent;    // see WgradArgs
};

struct Shared {
  uint64_t full[kStages];      // CTA 0: the stage's bytes of both CTAs landed (and were fixed)
  uint64_t empty[kStages];     // both: the MMAs finished reading the stage
  uint64_t landed[kStages];    // each CTA: its own bytes of a stage that needs fixing landed
  uint64_t acc_full[2];        // both: the buffer's tile is complete
  uint64_t acc_empty[2];       // CTA 0: both CTAs' epilogues have read it
  uint64_t drained;            // both
  uint32_t tmem_base;
  uint32_t sink;               // target of CTA 1's signalling stores (never read)
  uint32_t consumed;
  int abort_flag;
};
static_assert(sizeof(Shared) <= 512, "barrier block");

struct Unit {
  int g, mat, m0, n0, row0, rows;
  int tiles;  // 1 or 2
};
MOE_DEV Unit decode(const Params& p, int u) {
  Unit t{};
  if (u >= p.units) return t;
  t.g = u / p.units_per_group;
  int left = u - t.g * p.units_per_group;
  t.row0 = __ldg(p.grp_row0 + t.g);
  t.rows = __ldg(p.grp_rows + t.g);
  while (t.mat < p.nmat - 1 && left >= p.mat[t.mat].mt * p.mat[t.mat].nt) {
    left -= p.mat[t.mat].mt * p.mat[t.mat].nt;
    ++t.mat;
  }
  const Matrix& x = p.mat[t.mat];
  const int mi = left / x.nt, ni = left - mi * x.nt;
  t.m0 = mi * (x.split_m ? x.per_unit * kTile : kTile);
  t.n0 = ni * (x.split_m ? kTile : x.per_unit * kTile);
  t.tiles = x.per_unit == 2 && (x.split_m ? x.M - t.m0 : x.N - t.n0) > kTile ? 2 : 1;
  return t;
}
// Which accumulator buffers a unit takes: both, or the one whose turn it is.
// Every role replays the same sequence.
struct Buffers {
  uint32_t next = 0, uses[2] = {0u, 0u};
  uint32_t first = 0;
  MOE_DEV void take(int tiles) {
    first = tiles == 2 ? 0u : next;
    next = tiles == 2 ? 0u : next ^ 1u;
  }
  // parity of the phase of the buffer's next use
  MOE_DEV uint32_t parity(uint32_t b) const { return uses[b] & 1u; }
};
// A pair's units, u = pair, pair + pairs, ...: the next one is decoded while
// the current one is worked on (its two table reads and divisions cost about
// 900 cycles otherwise, in every role).
struct Walk {
  int u, step;
  Unit next;
  MOE_DEV Walk(const Params& p, int pair, int pairs) : u(pair), step(pairs), next(decode(p, pair)) {}
  MOE_DEV bool take(const Params& p, Unit& t) {
    if (u >= p.units) return false;
    t = next;
    u += step;
    next = decode(p, u);
    return true;
  }
};
// Rows of the last 64-row block, and whether foreign rows share its last K step.
MOE_DEV int tail_rows(int rows) { return rows - (rows - 1) / kBK * kBK; }

MOE_DEV void tma_store_3d(const void* tmap, uint32_t smem_src, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(smem_src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
// Adds the fp32 box to global memory (each element of dW is added to once).
MOE_DEV void tma_add_3d(const void* tmap, uint32_t smem_src, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(smem_src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

template <bool F32>
__global__ void __launch_bounds__(kThreads, 1) wgrad_tc_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_tiles = smem + kStages * kStageBytes;
  Shared& sh = *reinterpret_cast<Shared*>(out_tiles + kEpiWarps * kOutTile);
  const int warp = uniform_warp_id(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool first = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      // the first CTA's producer and the bytes of both CTAs, or (a fixed
      // stage) four bytes from each CTA's fixer
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
      mbar_init(&sh.landed[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.acc_full[b], 1);
      mbar_init(&sh.acc_empty[b], kEpiWarps);
    }
    mbar_init(&sh.drained, 1);
    sh.abort_flag = 0;
    sh.consumed = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (!p.independent) griddep_wait();
  Walk walk(p, (int)(blockIdx.x >> 1), (int)(gridDim.x >> 1));
  Unit t;
  Buffers buf;
  const uint32_t tmem_base = sh.tmem_base;
  volatile int* abort_flag = &sh.abort_flag;
  auto in_first = [&](const void* local) { return map_to_rank(smem_u32(local), 0u); };
  auto fail = [&]() {
    *abort_flag = 1;
    set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
  };

  uint32_t fills = 0, fixes = 0, fix_phase = 0;  // producer: fills issued; slots whose last fill is fixed; uses of landed[]
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      bool ok = true;
      while (ok && walk.take(p, t)) {
        if (t.rows == 0) continue;
        const Matrix& x = p.mat[t.mat];
        const int nk = (t.rows + kBK - 1) / kBK;
        const bool ragged = tail_rows(t.rows) % 16 != 0;
        // the shared operand's columns, and the first tile's own
        const CUtensorMap* ts = x.split_m ? &x.b : &x.a;
        const CUtensorMap* to = x.split_m ? &x.a : &x.b;
        const int cs = (x.split_m ? t.n0 : t.m0) + 128 * (int)rank, co = (x.split_m ? t.m0 : t.n0) + 128 * (int)rank;
        const uint32_t bytes = (1 + t.tiles) * kPart;
        for (int kc = 0; kc < nk; ++kc, ++fills) {
            const uint32_t s = fills % kStages;
            if (!mbar_wait_cluster_bounded(&sh.empty[s], ((fills / kStages) & 1u) ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            uint8_t* dst = smem + s * kStageBytes;
            const int r = t.row0 + kc * kBK;
            const bool fix = ragged && kc == nk - 1;
            if (fix) {
              // this CTA's bytes land on its own barrier; the fixers hand the stage on
              mbar_arrive_expect_tx(&sh.landed[s], bytes);
              if (first) mbar_arrive_expect_tx(&sh.full[s], 8);
              for (int c = 0; c < 2; ++c) tma_load_2d_hint(dst + c * kBox, ts, &sh.landed[s], cs + 64 * c, r, pol);
              for (int h = 0; h < t.tiles; ++h)
                for (int c = 0; c < 2; ++c)
                  tma_load_2d_hint(dst + (1 + h) * kPart + c * kBox, to, &sh.landed[s], co + kTile * h + 64 * c, r, pol);
              fixes |= 1u << s;
              fix_phase ^= 1u << s;
            } else {
              const uint32_t bar = in_first(&sh.full[s]);
              if (first) mbar_arrive_expect_tx(&sh.full[s], 2 * bytes);
              for (int c = 0; c < 2; ++c) tma_load_2d_pair(dst + c * kBox, ts, bar, cs + 64 * c, r, pol);
              for (int h = 0; h < t.tiles; ++h)
                for (int c = 0; c < 2; ++c)
                  tma_load_2d_pair(dst + (1 + h) * kPart + c * kBox, to, bar, co + kTile * h + 64 * c, r, pol);
              fixes &= ~(1u << s);
            }
          }
      }
      griddep_launch_dependents();
      if (!ok) fail();
    }
    __syncwarp();
  } else if (warp == 1) {
    if (first) {
      // the whole warp runs the loop, one elected lane issues
      const uint32_t idesc = idesc_bf16_f32(256, kTile) | kIdescAMn | kIdescBMn;
      uint32_t consumed = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu, mbar_wait_cluster_bounded(bar, parity, abort_flag));
        if (ok) tc_fence_after();
        return ok;
      };
      while (ok && walk.take(p, t)) {
        const int rows = __shfl_sync(0xffffffffu, t.rows, 0);
        const int tiles = __shfl_sync(0xffffffffu, t.tiles, 0);
        if (rows == 0) continue;
        const int nk = (rows + kBK - 1) / kBK;
        const int last_steps = (tail_rows(rows) + 15) / 16;
        // tile operands by shared-memory part: A and B are the shared part 0 or the tile's own
        const bool split_m = __shfl_sync(0xffffffffu, p.mat[t.mat].split_m, 0);
        buf.take(tiles);
        auto issue = [&](uint32_t j, int kc, int h, uint32_t b) {
          const uint64_t shared = smem_desc_sw128_mn(smem_u32(smem) + (j % kStages) * kStageBytes, kBox);
          const uint64_t own = shared + ((1 + h) * kPart >> 4);
          const uint64_t da = split_m ? own : shared, db = split_m ? shared : own;
          const int steps = kc == nk - 1 ? last_steps : kBK / 16;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            if (kk < steps)
              umma_bf16_pair(tmem_base + b * kTile, da + kk * (2048 >> 4), db + kk * (2048 >> 4), idesc, (kc | kk) != 0);
        };
        if (!wait(&sh.acc_empty[buf.first], buf.parity(buf.first) ^ 1u)) break;
        ++buf.uses[buf.first];
        const int lead = tiles == 2 ? (nk < kLead ? nk : kLead) : 0;
        for (int kc = 0; kc < lead; ++kc) {
          const uint32_t j = consumed + kc;
          if (!wait(&sh.full[j % kStages], (j / kStages) & 1u)) break;
          if (elect_one()) issue(j, kc, 0, 0);
          __syncwarp();
        }
        if (!ok) break;
        if (tiles == 2) {
          if (!wait(&sh.acc_empty[1], buf.parity(1) ^ 1u)) break;
          ++buf.uses[1];
        }
        for (int kc = 0; kc < nk; ++kc, ++consumed) {
          const uint32_t s = consumed % kStages;
          if (kc >= lead && !wait(&sh.full[s], (consumed / kStages) & 1u)) break;
          if (elect_one()) {
            if (kc >= lead) issue(consumed, kc, 0, buf.first);
            if (tiles == 2) issue(consumed, kc, 1, 1);
            umma_commit_pair_both(smem_u32(&sh.empty[s]));
          }
          __syncwarp();
        }
        if (ok && elect_one()) {
          umma_commit_pair_both(smem_u32(&sh.acc_full[buf.first]));
          if (tiles == 2) umma_commit_pair_both(smem_u32(&sh.acc_full[1]));
        }
        __syncwarp();
      }
      if (!ok && lane == 0) fail();
      if (elect_one()) umma_commit_pair_both(smem_u32(&sh.drained));
      if (lane == 0) sh.consumed = consumed;
      __syncwarp();
    }
    if (lane == 0) {
      int no_abort = 0;
      if (!mbar_wait_cluster_bounded(&sh.drained, 0, &no_abort)) set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
    }
    __syncwarp();
  } else if (warp < 2 + kEpiWarps) {
    const int q = warp & 3, ew = warp - 2, sub = ew >> 2;
    const uint32_t tile = smem_u32(out_tiles + ew * kOutTile);
    // this warp's half of a tile's columns in 128-byte tile rows: converted to
    // registers first, so that the buffer is free for the next MMAs before the stores
    constexpr int kCols = F32 ? 32 : 64, kBlocks = kTile / kCols / 2;
    while (walk.take(p, t)) {
      if (t.rows == 0 && p.accumulate) continue;
      const Matrix& x = p.mat[t.mat];
      if (t.rows > 0) {
        buf.take(t.tiles);
        int ok = 1;
        if (lane == 0)
          for (int h = 0; h < t.tiles && ok; ++h)
            ok = mbar_wait_cluster_bounded(&sh.acc_full[buf.first + h], buf.parity(buf.first + h), abort_flag);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) fail();
          break;
        }
        tc_fence_after();
      }
      const uint32_t t_q = tmem_base + ((uint32_t)(q * 32) << 16) + buf.first * kTile;
      uint32_t v[kBlocks][32];
      auto read = [&](int h, int i) {  // block i of tile h to registers
        const uint32_t at = t_q + h * kTile + (2 * i + sub) * kCols;
        if (t.rows == 0) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[i][j] = 0u;
        } else if (F32) {
          tmem_ld32(at, v[i]);
          tmem_wait_ld();
        } else {
          uint32_t w[32];
          tmem_ld32(at, v[i]);
          tmem_ld32(at + 32, w);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[i][j] = pack_bf16x2(__uint_as_float(v[i][2 * j]), __uint_as_float(v[i][2 * j + 1]));
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[i][16 + j] = pack_bf16x2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        }
      };
      auto release = [&](int h) {
        if (t.rows == 0) return;
        const uint32_t b = buf.first + h;
        ++buf.uses[b];
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!first) st_async_u32(in_first(&sh.sink), 0u, in_first(&sh.acc_empty[b]));
          else if (ew == 0) mbar_arrive_expect_tx(&sh.acc_empty[b], 4 * kEpiWarps);  // and CTA 1's warps' stores
          else mbar_arrive(&sh.acc_empty[b]);
        }
      };
      auto store = [&](int h, int i) {
        const int m = t.m0 + (x.split_m ? kTile * h : 0) + 128 * (int)rank + 32 * q;
        const int n = t.n0 + (x.split_m ? 0 : kTile * h) + (2 * i + sub) * kCols;
        if (m >= x.M || n >= x.N) return;
        if (lane == 0) bulk_wait_group_read<0>();  // the previous store has read the tile
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_v4(tile + lane * 128 + ((j ^ (lane & 7)) << 4),
                       make_uint4(v[i][4 * j], v[i][4 * j + 1], v[i][4 * j + 2], v[i][4 * j + 3]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (p.accumulate) tma_add_3d(&x.out, tile, n, m, t.g);
          else tma_store_3d(&x.out, tile, n, m, t.g);
          bulk_commit_group();
        }
      };
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) read(0, i);
      release(0);
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        store(0, i);
        if (t.tiles == 2) read(1, i);  // its registers are free again
      }
      if (t.tiles == 2) {
        release(1);
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) store(1, i);
      }
    }
    if (lane == 0) bulk_wait_group_all();
  } else {
    // ------------------------------------------------------------- fixer --
    uint32_t j = 0, phase = 0;
    bool ok = true;
    while (ok && walk.take(p, t)) {
      if (t.rows == 0) continue;
      const int nk = (t.rows + kBK - 1) / kBK;
      const int v = tail_rows(t.rows);
      j += nk;
      if (v % 16 == 0) continue;
      {
        const uint32_t s = (j - 1) % kStages;
        int got = 1;
        if (lane == 0) got = mbar_wait_bounded(&sh.landed[s], (phase >> s) & 1u, abort_flag);
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          if (lane == 0) fail();
          ok = false;
          break;
        }
        phase ^= 1u << s;
        // rows v .. (the next multiple of 16) - 1 of the four or six boxes, 128 bytes each
        const uint32_t at = smem_u32(smem + s * kStageBytes);
        for (int r = v; r & 15; ++r) {
          const uint32_t row = at + (lane >> 3) * kBox + r * 128 + (lane & 7) * 16;
          st_shared_v4(row, make_uint4(0, 0, 0, 0));
          if (t.tiles == 2 && lane < 16) st_shared_v4(row + 4 * kBox, make_uint4(0, 0, 0, 0));
        }
        fence_proxy_async_smem();
        __syncwarp();
        // (an asynchronous store: a remote arrive would hold this warp for about 1000 cycles)
        if (lane == 0) st_async_u32(in_first(&sh.sink), 0u, in_first(&sh.full[s]));
      }
    }
  }

  __syncthreads();
  if (warp == 0 && lane == 0) {
    // wait for any stage fill that was issued but may not have landed
    const uint32_t done = first ? sh.consumed : (fills > kStages ? fills - kStages : 0u);
    for (uint32_t j = done; j < fills; ++j) {
      const uint32_t s = j % kStages;
      int no_abort = 0;
      const bool fixed = (fixes >> s) & 1u;
      if (!fixed && !first) continue;  // the first CTA's barrier: waited for there
      if (!(fixed ? mbar_wait_bounded(&sh.landed[s], ((fix_phase >> s) & 1u) ^ 1u, &no_abort)
                  : mbar_wait_cluster_bounded(&sh.full[s], (j / kStages) & 1u, &no_abort))) {
        set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
        break;
      }
    }
  }
  if (p.independent) griddep_wait();  // this grid ends after its predecessor
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still touch its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

bool make_rows_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, stride[1] = {(uint64_t)ld * 2};
  const uint32_t box[2] = {64, kBK};
  return make_tmap_nd(m, base, 2, 2, dims, stride, box, 128, true);
}

}  // namespace

cudaError_t launch_wgrad_tc(const WgradArgs& a, cudaStream_t s) {
  Params p{};
  p.nmat = a.nmat;
  p.groups = a.groups;
  const int elem = a.grad_dtype == MOE_F32 ? 4 : 2;
  for (int i = 0; i < a.nmat; ++i) {
    const WgradMatrix& w = a.mat[i];
    Matrix& x = p.mat[i];
    x.M = (int)w.M;
    x.N = w.N;
    // Two tiles side by side, along the dimension with an even number of them
    // (all units then have two) or else along the longer one -- unless there
    // are so few tiles that the coarser units leave pairs idle: a unit of two
    // takes about 1.6 times a unit of one.
    const int64_t tm = (w.M + kTile - 1) / kTile, tn = (w.N + kTile - 1) / kTile;
    x.split_m = tm % 2 == tn % 2 ? tm >= tn : tm % 2 == 0;
    const int64_t one = tm * tn, two = x.split_m ? (tm + 1) / 2 * tn : tm * ((tn + 1) / 2);
    const int64_t pairs = device_sm_count() / 2;
    auto rounds = [&](int64_t units) { return (units * a.groups + pairs - 1) / pairs; };
    x.per_unit = 10 * rounds(one) <= 16 * rounds(two) ? 1 : 2;
    x.mt = (int)(x.split_m ? (tm + x.per_unit - 1) / x.per_unit : tm);
    x.nt = (int)(x.split_m ? tn : (tn + x.per_unit - 1) / x.per_unit);
    p.units_per_group += x.mt * x.nt;
    const uint64_t dims[3] = {(uint64_t)w.N, (uint64_t)w.M, (uint64_t)a.groups};
    const uint64_t stride[2] = {(uint64_t)w.N * elem, (uint64_t)w.N * w.M * elem};
    const uint32_t box[3] = {128u / elem, 32, 1};
    if (!make_rows_map(&x.a, w.A, a.rows, w.M, w.lda) || !make_rows_map(&x.b, w.B, a.rows, w.N, w.N) ||
        !make_tmap_nd(&x.out, w.out, elem, 3, dims, stride, box, 128, false))
      return cudaErrorInvalidValue;
  }
  const int64_t units = (int64_t)a.groups * p.units_per_group;
  if (units > (1ll << 31) - 1 - 4096) return cudaErrorInvalidValue;
  p.units = (int)units;
  p.grp_row0 = a.grp_row0;
  p.grp_rows = a.grp_rows;
  p.accumulate = a.accumulate;
  p.status = a.status;
  p.independent = a.independent;
  if (p.units == 0) return cudaSuccess;

  const bool f32 = a.grad_dtype == MOE_F32;
  const auto kernel = f32 ? wgrad_tc_kernel<true> : wgrad_tc_kernel<false>;
  static std::mutex mu;
  static int max_clusters_of[2][kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    int& known = max_clusters_of[f32][dev];
    if (known == 0) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      cfg.gridDim = dim3(2 * (device_sm_count() / 2), 1, 1);
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (e != cudaSuccess) return e;
      known = n > 0 ? n : 1;
    }
    clusters = known;
  }
  if (p.units < clusters) clusters = p.units;
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_route_products_tc(const Problem& p, const RouteBwdArgs& a, cudaStream_t s) {
  if (a.dx) {
    WgradArgs x{};
    x.mat[0] = {a.dz16_t, a.W_r, a.dx, p.T, p.d, a.ld_t};
    x.nmat = 1;
    x.groups = 1;
    x.rows = p.N;
    x.grp_row0 = a.tables + kRtRow0;
    x.grp_rows = a.tables + kRtExperts;
    x.grad_dtype = MOE_BF16;
    x.status = a.status;
    const cudaError_t e = launch_wgrad_tc(x, s);
    if (e != cudaSuccess) return e;
  }
  if (!a.dW_r) return cudaSuccess;
  const bool split = a.splits > 1;
  WgradArgs w{};
  w.mat[0] = {a.dz16, a.x, split ? a.planes : a.dW_r, p.N, p.d, a.ld};
  w.nmat = 1;
  w.groups = a.splits;
  w.rows = p.T;
  w.grp_row0 = a.tables + kRtSplit0;
  w.grp_rows = a.tables + kRtSplitRows;
  w.grad_dtype = split ? (int)MOE_F32 : a.grad_dtype;
  w.accumulate = !split && a.accumulate;
  w.status = a.status;
  w.independent = a.dx != nullptr;  // of the dx product, which has waited for dz
  const cudaError_t e = launch_wgrad_tc(w, s);
  if (e != cudaSuccess || !split) return e;
  return launch_join_planes(a.planes, a.splits, (int64_t)p.N * p.d, a.dW_r, a.grad_dtype, a.accumulate, s);
}

}  // namespace moe
