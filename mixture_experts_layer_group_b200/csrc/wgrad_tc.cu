// Weight gradients on the tensor cores: dW[g][m][n] = sum over the rows r of
// group g of A[r][m] B[r][n], for several matrices in one launch (the
// experts' dW1 = dg^T x, dW3 = du^T x, dW2 = dy^T (gate h); the router's
// dW_r = dz^T x, and its dx = (dz^T)^T W_r over the experts as rows). Both
// operands are row-major with the rows as the reduction, so both are MN-major
// tiles: a 64 x 64 TMA box is 64 rows (k) of 128 bytes.
//
// CTA pairs (clusters of 2, cta_group::2): a unit is a run of 256 x 256 tiles
// of one group's matrix that share an operand (side by side along M or along
// N). CTA r loads 128 of the 256 columns of either operand per 64 rows -- a
// piece of 16 KB, twelve of which are its shared memory, some for the shared
// operand, the rest for the tiles' own -- and keeps rows 128 r .. 128 r + 127
// of a tile in its tensor memory, in one of two 256-column buffers.
//
// What bounds long sums is the operands' way from L2 (the SMs took 29 bytes per
// cycle each on average, with the tensor pipe 60 % busy), and short ones the
// writing of the result, so a unit reuses the shared operand as its rows allow:
//   few rows (the shared operand's pieces hold them all): it is loaded once for
//     the whole run, and each tile streams its own operand past it, 32 KB per
//     pair and 512 cycles of pair MMAs; tiles alternate between the buffers
//   many rows: the tiles go in twos, both fed by one pass over the rows, 96 KB
//     per 1024 cycles; between two passes the first tile's MMAs of two stages run
//     while the second tile is still being read
// One tile at a time would take 64 KB per 512 cycles. Measured: the gradients of
// 63 experts of 896 x 1280 over 57344 rows 350 us (395 GFLOP, 1.13 PFLOP/s), of
// one of 2048 x 7168 over 4096 rows 247 us (1.46 PFLOP/s), of 32 of those over
// 8192 rows 746 us: 2.8 GB written, 724 us at the 3.89 TB/s that a B200 writes
// when it does nothing else. (The whole backward with tiles one by one: 946, 598
// and 1622 us, in twos 911, 563 and 1548.)
//
// A group's last piece may hold up to 15 rows of the next group inside its
// last K = 16 step. They would enter the sum, and a NaN there cannot be
// multiplied away, so a fixer warp in each CTA zeroes them in both operands
// before the piece is handed to the MMA issuer.
//
// Warps: 0 producer of the shared operand, 1 tensor-memory owner and MMA issuer
// (first CTA), 2..9 epilogue (two per lane quadrant), 10 fixer, 11 producer of the
// tiles' own operands. A producer needs about 300 cycles for a piece (the wait
// for its slot, the barrier's expected bytes) and 30 for each box; one warp for
// both operands would fall behind the MMAs. Every role replays the same walk
// over units, pieces and buffers. Waits are bounded as everywhere.
#include <initializer_list>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kBK = 64;
constexpr int kTile = 256;
constexpr int kBox = 64 * kBK * 2;           // 8 KB
constexpr int kPiece = 2 * kBox;             // 128 columns x 64 rows of an operand
constexpr int kPieces = 12;
constexpr int kLead = 2;                     // stages whose second tile follows later at the start of a pass
constexpr int kMaxRun = 8;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kOutTile = 32 * 128;           // 32 rows x 128 bytes per epilogue warp
constexpr int kSmem = kPieces * kPiece + kEpiWarps * kOutTile + 1024 + 512;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kTmemCols = 512;

struct Matrix {
  CUtensorMap a;    // [R, M]
  CUtensorMap b;    // [R, N]
  CUtensorMap out;  // [groups, M, N]
  int M, N, mt, nt;  // units along M and N
  int split_m;       // a unit's tiles lie along M (else along N)
  int run;           // tiles of a unit at most
  // a piece of A (B) is one box: the map is [columns / 64][rows][64]; otherwise
  // (columns no multiple of 64) two boxes of a [rows][columns] map
  int whole_a, whole_b;
};
struct Params {
  Matrix mat[3];
  int nmat, groups;
  int units_per_group, units;
  int shared_pieces;  // of the kPieces, for the shared operand
  const int32_t* grp_row0;
  const int32_t* grp_rows;
  int accumulate;
  unsigned* status;
  const int* ready;  // see WgradArgs
  int* publish;
  int beside;
};

struct Shared {
  uint64_t full[kPieces];      // CTA 0: the piece's bytes of both CTAs landed (and were fixed)
  uint64_t empty[kPieces];     // both: the MMAs finished reading the piece
  uint64_t landed[kPieces];    // each CTA: its own bytes of a piece that needs fixing landed
  uint64_t acc_full[2];        // both: the buffer's tile is complete
  uint64_t acc_empty[2];       // CTA 0: both CTAs' epilogues have read it
  uint64_t drained;            // both
  uint32_t tmem_base;
  uint32_t sink;               // target of CTA 1's signalling stores (never read)
  int abort_flag;
  int go;                      // what is read may be read
};
static_assert(sizeof(Shared) <= 512, "barrier block");

struct Unit {
  int g, mat, m0, n0, row0, rows;
  int tiles;
  // the same values, in a form the compiler keeps in uniform registers
  MOE_DEV void uniform() {
    for (int* v : {&g, &mat, &m0, &n0, &row0, &rows, &tiles}) *v = __shfl_sync(0xffffffffu, *v, 0);
  }
};
MOE_DEV Unit decode(const Params& p, int u) {
  Unit t{};
  if (u >= p.units) return t;
  t.g = u / p.units_per_group;
  int left = u - t.g * p.units_per_group;
  t.row0 = ld_after_wait(p.grp_row0 + t.g);
  t.rows = ld_after_wait(p.grp_rows + t.g);
  while (t.mat < p.nmat - 1 && left >= p.mat[t.mat].mt * p.mat[t.mat].nt) {
    left -= p.mat[t.mat].mt * p.mat[t.mat].nt;
    ++t.mat;
  }
  const Matrix& x = p.mat[t.mat];
  const int mi = left / x.nt, ni = left - mi * x.nt;
  t.m0 = mi * (x.split_m ? x.run * kTile : kTile);
  t.n0 = ni * (x.split_m ? kTile : x.run * kTile);
  const int span = x.split_m ? x.M - t.m0 : x.N - t.n0;
  t.tiles = span >= x.run * kTile ? x.run : (span + kTile - 1) / kTile;
  return t;
}
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
// A position in one operand's pieces: slots first .. first + count - 1 in turn.
struct Cursor {
  int slot, first, count;
  uint32_t phase = 0;  // parity of the slot's current use
  MOE_DEV Cursor(int f, int n) : slot(f), first(f), count(n) {}
  MOE_DEV void next() {
    if (++slot == first + count) {
      slot = first;
      phase ^= 1u;
    }
  }
};
// Which accumulator buffers a pass takes: both for two tiles, or the one whose
// turn it is.
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
// Rows of the last 64-row piece; foreign rows share its last K step unless
// they are a multiple of 16.
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
  uint8_t* out_tiles = smem + kPieces * kPiece;
  Shared& sh = *reinterpret_cast<Shared*>(out_tiles + kEpiWarps * kOutTile);
  const int warp = uniform_warp_id(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool first = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPieces; ++s) {
      // the first CTA's producer and the bytes of both CTAs, or (a fixed
      // piece) four bytes from each CTA's fixer
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
    fence_barrier_init();
  }
  if (threadIdx.x == 64) {
    sh.go = !p.ready || take_published(p.ready);
    if (!sh.go) set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
  }
  if (warp == 1) {
    tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (!p.ready) griddep_wait();
  else fence_proxy_async_global();
  // (the vote keeps what follows warp-uniform for the compiler: read as it is, the flag
  // moved the walks out of uniform registers, 154 -> 168 of them and spills)
  if (!__any_sync(0xffffffffu, sh.go)) {  // nothing may be read; the waits of the other CTA run out
    griddep_wait();
    cluster_sync();
    if (warp == 1) tmem_dealloc_pair(sh.tmem_base, kTmemCols);
    return;
  }
  if (threadIdx.x == 64) {  // (not a producer: the release takes about 1 us)
    if (p.publish && blockIdx.x == 0) publish_waited(p.publish);
    if (p.beside) griddep_launch_dependents();
  }
  Walk walk(p, (int)(blockIdx.x >> 1), (int)(gridDim.x >> 1));
  Unit t;
  Buffers buf;
  // pieces of the shared operand and of the tiles' own
  Cursor cs(0, p.shared_pieces), co(p.shared_pieces, kPieces - p.shared_pieces);
  const int most_kept = p.shared_pieces;  // pieces of the shared operand that can stay for a whole run
  const uint32_t tmem_base = sh.tmem_base;
  volatile int* abort_flag = &sh.abort_flag;
  auto in_first = [&](const void* local) { return map_to_rank(smem_u32(local), 0u); };
  auto fail = [&]() {
    *abort_flag = 1;
    set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
  };

  // producers: pieces whose last load went to landed[], uses of landed[], and pieces loaded at all
  uint32_t fixes = 0, fix_phase = 0, loaded = 0, load_phase = 0;
  if (warp == 0 || warp == 3 + kEpiWarps) {
    {
      const bool for_shared = warp == 0;
      // the whole warp runs the loop, one elected lane issues (see elect_one())
      const uint64_t pol = policy_evict_normal();
      bool ok = true;
      // one piece: columns c of a map's rows r, into the cursor's slot
      auto load = [&](Cursor& at, const CUtensorMap* map, bool whole, int c, int r, bool fix) {
        const int s = at.slot;
        ok = __all_sync(0xffffffffu, mbar_wait_cluster_bounded(&sh.empty[s], at.phase ^ 1u, abort_flag));
        if (!ok) return;
        uint8_t* dst = smem + s * kPiece;
        const uint32_t bit = 1u << s;
        if (fix) {
          // this CTA's bytes land on its own barrier; the fixers hand the piece on
          if (elect_one()) {
            mbar_arrive_expect_tx(&sh.landed[s], kPiece);
            if (first) mbar_arrive_expect_tx(&sh.full[s], 8);
            if (whole) {
              tma_load_3d_hint(dst, map, &sh.landed[s], 0, r, c >> 6, pol);
            } else {
              tma_load_2d_hint(dst, map, &sh.landed[s], c, r, pol);
              tma_load_2d_hint(dst + kBox, map, &sh.landed[s], c + 64, r, pol);
            }
          }
          fixes |= bit;
          fix_phase ^= bit;
        } else {
          const uint32_t bar = in_first(&sh.full[s]);
          if (elect_one()) {
            if (first) mbar_arrive_expect_tx(&sh.full[s], 2 * kPiece);
            if (whole) {
              tma_load_3d_pair(dst, map, bar, 0, r, c >> 6, pol);
            } else {
              tma_load_2d_pair(dst, map, bar, c, r, pol);
              tma_load_2d_pair(dst + kBox, map, bar, c + 64, r, pol);
            }
          }
          fixes &= ~bit;
        }
        __syncwarp();
        loaded |= bit;
        load_phase = at.phase ? load_phase | bit : load_phase & ~bit;
        at.next();
      };
      while (ok && walk.take(p, t)) {
        t.uniform();
        if (t.rows == 0) continue;
        const Matrix& x = p.mat[t.mat];
        const int nk = (t.rows + kBK - 1) / kBK;
        const bool ragged = tail_rows(t.rows) % 16 != 0;
        const bool keep = nk <= most_kept, is_a = for_shared != (bool)x.split_m;
        const CUtensorMap* map = is_a ? &x.a : &x.b;
        const bool whole = is_a ? x.whole_a : x.whole_b;
        const int c = (is_a ? t.m0 : t.n0) + 128 * (int)rank;
        Cursor& at = for_shared ? cs : co;
        for (int h = 0; h < t.tiles && ok; h += keep ? 1 : 2) {
          if (for_shared && keep && h > 0) break;
          const int own = keep || for_shared || h + 1 == t.tiles ? 1 : 2;
          for (int kc = 0; kc < nk && ok; ++kc)
            for (int i = 0; i < own && ok; ++i)
              load(at, map, whole, for_shared ? c : c + kTile * (h + i), t.row0 + kc * kBK, ragged && kc == nk - 1);
        }
      }
      if (for_shared && elect_one()) griddep_launch_dependents();
      if (!ok && lane == 0) fail();
    }
    __syncwarp();
  } else if (warp == 1) {
    if (first) {
      // the whole warp runs the loop, one elected lane issues
      const uint32_t idesc = idesc_bf16_f32(256, kTile) | kIdescAMn | kIdescBMn;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu, mbar_wait_cluster_bounded(bar, parity, abort_flag));
        if (ok) tc_fence_after();
        return ok;
      };
      while (ok && walk.take(p, t)) {
        t.uniform();
        const int rows = t.rows, tiles = t.tiles;
        if (rows == 0) continue;
        const int nk = (rows + kBK - 1) / kBK;
        const int last_steps = (tail_rows(rows) + 15) / 16;
        // is the shared operand B (its tiles lie along M) or A?
        const bool split_m = p.mat[t.mat].split_m;
        // the MMAs of one stage of one tile into buffer b
        auto issue = [&](int shared_slot, int own_slot, int kc, uint32_t b) {
          const uint64_t ds = smem_desc_sw128_mn(smem_u32(smem) + shared_slot * kPiece, kBox);
          const uint64_t dn = smem_desc_sw128_mn(smem_u32(smem) + own_slot * kPiece, kBox);
          const uint64_t da = split_m ? dn : ds, db = split_m ? ds : dn;
          const int steps = kc == nk - 1 ? last_steps : kBK / 16;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            if (kk < steps)
              umma_bf16_pair(tmem_base + b * kTile, da + kk * (2048 >> 4), db + kk * (2048 >> 4), idesc, (kc | kk) != 0);
        };
        auto done = [&](int slot) { umma_commit_pair_both(smem_u32(&sh.empty[slot])); };
        if (nk <= most_kept) {
          for (int h = 0; h < tiles && ok; ++h) {
            buf.take(1);
            const uint32_t b = buf.first;
            if (!wait(&sh.acc_empty[b], buf.parity(b) ^ 1u)) break;
            ++buf.uses[b];
            Cursor s = cs;
            for (int kc = 0; kc < nk; ++kc) {
              if (h == 0 && !wait(&sh.full[s.slot], s.phase)) break;
              if (!wait(&sh.full[co.slot], co.phase)) break;
              if (elect_one()) {
                issue(s.slot, co.slot, kc, b);
                done(co.slot);
                if (h == tiles - 1) done(s.slot);
              }
              __syncwarp();
              s.next();
              co.next();
            }
            if (ok && elect_one()) umma_commit_pair_both(smem_u32(&sh.acc_full[b]));
            __syncwarp();
          }
          for (int kc = 0; kc < nk; ++kc) cs.next();
          continue;
        }
        for (int h = 0; h < tiles && ok; h += 2) {
          const int own = h + 1 == tiles ? 1 : 2;
          buf.take(own);
          const uint32_t b0 = buf.first;
          if (!wait(&sh.acc_empty[b0], buf.parity(b0) ^ 1u)) break;
          ++buf.uses[b0];
          // (a pass of two tiles: their own pieces alternate)
          const int lead = own == 2 ? (nk < kLead ? nk : kLead) : 0;
          Cursor s = cs, n = co;
          for (int kc = 0; kc < lead; ++kc) {
            if (!wait(&sh.full[s.slot], s.phase) || !wait(&sh.full[n.slot], n.phase)) break;
            if (elect_one()) {
              issue(s.slot, n.slot, kc, 0);
              done(n.slot);
            }
            __syncwarp();
            s.next();
            n.next();
            n.next();
          }
          if (!ok) break;
          if (own == 2) {
            if (!wait(&sh.acc_empty[1], buf.parity(1) ^ 1u)) break;
            ++buf.uses[1];
          }
          for (int kc = 0; kc < nk; ++kc) {
            if (kc >= lead) {
              if (!wait(&sh.full[cs.slot], cs.phase) || !wait(&sh.full[co.slot], co.phase)) break;
              if (elect_one()) {
                issue(cs.slot, co.slot, kc, b0);
                done(co.slot);
              }
              __syncwarp();
            }
            co.next();
            if (own == 2 && !wait(&sh.full[co.slot], co.phase)) break;
            if (elect_one()) {
              if (own == 2) {
                issue(cs.slot, co.slot, kc, 1);
                done(co.slot);
              }
              done(cs.slot);
            }
            __syncwarp();
            if (own == 2) co.next();
            cs.next();
          }
          if (ok && elect_one()) {
            umma_commit_pair_both(smem_u32(&sh.acc_full[b0]));
            if (own == 2) umma_commit_pair_both(smem_u32(&sh.acc_full[1]));
          }
          __syncwarp();
        }
      }
      if (!ok && lane == 0) fail();
      if (elect_one()) umma_commit_pair_both(smem_u32(&sh.drained));
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
    bool ok = true;
    while (ok && walk.take(p, t)) {
      if (t.rows == 0 && p.accumulate) continue;
      const Matrix& x = p.mat[t.mat];
      const bool twos = t.rows > 0 && (t.rows + kBK - 1) / kBK > most_kept;
      for (int h0 = 0; h0 < t.tiles; h0 += twos ? 2 : 1) {
        const int tiles = twos && h0 + 1 < t.tiles ? 2 : 1;
        if (t.rows > 0) {
          buf.take(tiles);
          int got = 1;
          if (lane == 0)
            for (int h = 0; h < tiles && got; ++h)
              got = mbar_wait_cluster_bounded(&sh.acc_full[buf.first + h], buf.parity(buf.first + h), abort_flag);
          ok = __shfl_sync(0xffffffffu, got, 0);
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
          const int m = t.m0 + (x.split_m ? kTile * (h0 + h) : 0) + 128 * (int)rank + 32 * q;
          const int n = t.n0 + (x.split_m ? 0 : kTile * (h0 + h)) + (2 * i + sub) * kCols;
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
          if (tiles == 2) read(1, i);  // its registers are free again
        }
        if (tiles == 2) {
          release(1);
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) store(1, i);
        }
      }
    }
    if (lane == 0) bulk_wait_group_all();
  } else {
    // ------------------------------------------------------------- fixer --
    uint32_t phase = 0;
    bool ok = true;
    auto fix = [&](int s, int v) {  // zero rows v .. (the next multiple of 16) - 1 of the piece's two boxes
      int got = 1;
      if (lane == 0) got = mbar_wait_bounded(&sh.landed[s], (phase >> s) & 1u, abort_flag);
      ok = __shfl_sync(0xffffffffu, got, 0);
      if (!ok) {
        if (lane == 0) fail();
        return;
      }
      phase ^= 1u << s;
      const uint32_t at = smem_u32(smem + s * kPiece) + ((lane >> 3) & 1) * kBox + (lane & 7) * 16;
      for (int r = v + (lane >> 4); r < (v + 15) / 16 * 16; r += 2) st_shared_v4(at + r * 128, make_uint4(0, 0, 0, 0));
      fence_proxy_async_smem();
      __syncwarp();
      // (an asynchronous store: a remote arrive would hold this warp for about 1000 cycles)
      if (lane == 0) st_async_u32(in_first(&sh.sink), 0u, in_first(&sh.full[s]));
    };
    while (ok && walk.take(p, t)) {
      if (t.rows == 0) continue;
      const int nk = (t.rows + kBK - 1) / kBK;
      const int v = tail_rows(t.rows);
      const bool keep = nk <= most_kept, ragged = v % 16 != 0;
      for (int h = 0; h < t.tiles && ok; h += keep ? 1 : 2) {
        const int own = keep || h + 1 == t.tiles ? 1 : 2;
        for (int kc = 0; kc < nk && ok; ++kc) {
          const bool last = ragged && kc == nk - 1;
          if (!keep || h == 0) {
            if (last) fix(cs.slot, v);
            cs.next();
          }
          for (int i = 0; i < own && ok; ++i) {
            if (last) fix(co.slot, v);
            co.next();
          }
        }
      }
    }
  }

  __syncthreads();
  if ((warp == 0 || warp == 3 + kEpiWarps) && lane == 0) {
    // wait for every piece's last load: it may not have landed when a wait gave up
    for (int s = 0; s < kPieces; ++s) {
      int no_abort = 0;
      const bool fixed = (fixes >> s) & 1u;
      if (!((loaded >> s) & 1u) || (!fixed && !first)) continue;  // not the first CTA: its barrier is waited for there
      if (!(fixed ? mbar_wait_bounded(&sh.landed[s], ((fix_phase >> s) & 1u) ^ 1u, &no_abort)
                  : mbar_wait_cluster_bounded(&sh.full[s], (load_phase >> s) & 1u, &no_abort))) {
        set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
        break;
      }
    }
  }
  if (p.ready) griddep_wait();  // this grid ends after its predecessor
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still touch its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// An operand's map: boxes of 64 columns x 64 rows, or, where the columns are a
// multiple of 64, two of them side by side as one box.
bool make_rows_map(CUtensorMap* m, int* whole, const void* base, int64_t rows, int64_t cols, int64_t ld) {
  *whole = cols % 64 == 0;
  if (*whole) {
    const uint64_t dims[3] = {64, (uint64_t)rows, (uint64_t)cols / 64}, stride[2] = {(uint64_t)ld * 2, 128};
    const uint32_t box[3] = {64, kBK, 2};
    return make_tmap_nd(m, base, 2, 3, dims, stride, box, 128, true);
  }
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, stride[1] = {(uint64_t)ld * 2};
  const uint32_t box[2] = {64, kBK};
  return make_tmap_nd(m, base, 2, 2, dims, stride, box, 128, true);
}

// The units of one matrix: runs of tiles along one dimension.
void choose_runs(Matrix& x, int64_t M, int N, int groups, bool keep, int64_t pairs) {
  x.M = (int)M;
  x.N = N;
  const int64_t tm = (M + kTile - 1) / kTile, tn = (N + kTile - 1) / kTile;
  auto units = [&](bool along_m, int run) {
    return (along_m ? (tm + run - 1) / run * tn : tm * ((tn + run - 1) / run)) * groups;
  };
  // Two tiles per unit: along the dimension with an even number of them (all
  // units then have two) or else along the longer one. With more (the shared
  // operand is kept): along the longer one.
  x.split_m = keep || tm % 2 == tn % 2 ? tm >= tn : tm % 2 == 0;
  // The run whose rounds over the CTA pairs cost least: a tile costs 10, its
  // share of the shared operand's loads 6 (as measured for one tile against two
  // per unit in long sums; in short ones the loads bind just the same).
  int64_t best = -1;
  for (int run = 1; run <= (keep ? kMaxRun : 2); ++run) {
    const int64_t rounds = (units(x.split_m, run) + pairs - 1) / pairs, cost = rounds * (10 * run + 6);
    if (best < 0 || cost < best) {
      best = cost;
      x.run = run;
    }
  }
  x.mt = (int)(x.split_m ? (tm + x.run - 1) / x.run : tm);
  x.nt = (int)(x.split_m ? tn : (tn + x.run - 1) / x.run);
}

}  // namespace

cudaError_t launch_wgrad_tc(const WgradArgs& a, cudaStream_t s) {
  Params p{};
  p.nmat = a.nmat;
  p.groups = a.groups;
  const int elem = a.grad_dtype == MOE_F32 ? 4 : 2;
  // Half of the pieces for the shared operand, when the groups' rows fit them
  // on average (384); otherwise a third, two pieces of the tiles' own to one of it.
  const bool keep = a.rows <= (int64_t)a.groups * (kPieces / 2) * kBK;
  p.shared_pieces = keep ? kPieces / 2 : kPieces / 3;
  for (int i = 0; i < a.nmat; ++i) {
    const WgradMatrix& w = a.mat[i];
    Matrix& x = p.mat[i];
    choose_runs(x, w.M, w.N, a.groups, keep, a.max_pairs > 0 ? a.max_pairs : device_sm_count() / 2);
    p.units_per_group += x.mt * x.nt;
    const uint64_t dims[3] = {(uint64_t)w.N, (uint64_t)w.M, (uint64_t)a.groups};
    const uint64_t stride[2] = {(uint64_t)w.N * elem, (uint64_t)w.N * w.M * elem};
    const uint32_t box[3] = {128u / elem, 32, 1};
    if (!make_rows_map(&x.a, &x.whole_a, w.A, a.rows, w.M, w.lda) ||
        !make_rows_map(&x.b, &x.whole_b, w.B, a.rows, w.N, w.N) ||
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
  p.ready = a.ready;
  p.publish = a.publish;
  p.beside = a.beside;
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
  if (a.max_pairs > 0 && a.max_pairs < clusters) clusters = a.max_pairs;
  if (p.units < clusters) clusters = p.units;
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// dW_r is N x d summed over all tokens, few tiles with a long sum; dx is T x d
// summed over the experts, many tiles with a short one. Run beside each other the
// two hide each other's fixed costs (launch, first loads, last stores), and where
// that leaves dW_r one token range its planes and their join are saved as well. In
// tenths of a microsecond, as measured: a tile of dx 24 (of 63 to 256 experts: most of it
// is the store and fixed costs, so fewer or more experts are priced alike), 64 tokens of a
// tile of dW_r 7, joining planes 50, and 60 before the second of two launches one
// after the other ends its first loads. The whole router backward, one after the other
// and beside: T 4096, N 256, d 7168 58 and 48; T 8192, N 63, d 1280 40 and 34; T 512,
// N 256, d 7168 33 and 22 us (without the flag between them, which adds up to 1 us).
// These three shapes are all that the prices were held against.
RoutePlan plan_route_products(const Problem& p) {
  const int64_t pairs = device_sm_count() / 2, column_tiles = (p.d + kTile - 1) / kTile;
  const int64_t dw_tiles = (p.N + kTile - 1) / kTile * column_tiles, dx_tiles = (p.T + kTile - 1) / kTile * column_tiles;
  int64_t most = pairs / dw_tiles;
  if (most > p.T / kTile) most = p.T / kTile;
  if (most > kMaxRouteSplits) most = kMaxRouteSplits;
  if (most < 1) most = 1;
  RoutePlan best{1, (int)most, 0};
  int64_t least = -1;
  for (int64_t n = 1; n <= most; ++n) {
    const int64_t rounds = (dw_tiles * n + pairs - 1) / pairs;
    const int64_t dw = rounds * ((p.T + 64 * n - 1) / (64 * n)) * 7, join = n > 1 ? 50 : 0;
    const int64_t after = (dx_tiles + pairs - 1) / pairs * 24 + 60 + dw + join;
    if (least < 0 || after < least) least = after, best.splits = (int)n, best.dx_pairs = 0;
    const int64_t left = pairs - dw_tiles * n;
    if (left <= 0) continue;
    const int64_t dx = (dx_tiles + left - 1) / left * 24, beside = (dx > dw ? dx : dw) + join;
    if (beside < least) least = beside, best.splits = (int)n, best.dx_pairs = (int)left;
  }
  return best;
}

cudaError_t launch_route_products_tc(const Problem& p, const RouteBwdArgs& a, cudaStream_t s) {
  const int dx_pairs = a.dx && a.dW_r ? plan_route_products(p).dx_pairs : 0;
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
    x.max_pairs = dx_pairs;
    x.publish = a.dW_r ? a.tables + kRtReady : nullptr;
    x.beside = dx_pairs > 0;
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
  w.ready = a.dx ? a.tables + kRtReady : nullptr;  // the dx product has waited for dz
  w.max_pairs = dx_pairs > 0 ? device_sm_count() / 2 - dx_pairs : 0;
  const cudaError_t e = launch_wgrad_tc(w, s);
  if (e != cudaSuccess || !split) return e;
  return launch_join_planes(a.planes, a.splits, (int64_t)p.N * p.d, a.dW_r, a.grad_dtype, a.accumulate, s);
}

}  // namespace moe
