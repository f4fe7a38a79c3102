// fp32 matrix products on CUDA cores: tiles of C[m, n] = sum_k A(m, k) B(n, k)
// with operands contiguous along either index, for the layers stored in fp32
// (tensor cores would round the operands to TF32). 256 threads.
//
// Sums are taken in two levels: chains of kChain fused multiply-adds over
// ascending k, and the chains' sums added up in order. One chain of 4096 terms is
// off by 1.1e-6 of the result (rms), in two levels by 2.3e-7. The order depends on
// the tile's shape alone, so results are the same each time.
#pragma once

#include "common.cuh"

namespace moe {
namespace simt {

constexpr int kThreads = 256;
constexpr int kChain = 128;

// A strided operand: element (r, k) at p[r * rs + k * ks] for r < rows and
// k < len, zero elsewhere. One of the strides is 1, the other and the bound
// along the unit stride are multiples of 4, so four consecutive elements load
// as one aligned vector.
struct Operand {
  const float* p;
  int64_t rs, ks;
  int rows, len;
};

// Column r of row k in a [k][rows] block: the 16-byte column groups of row k
// are permuted by k / 4, so that the four rows a k-contiguous vector is spread
// over, and the reads along a row, fall on different banks.
template <int ROWS>
MOE_DEV int swz(int k, int r) { return r ^ (((k >> 2) & (ROWS >= 32 ? 7 : ROWS / 4 - 1)) << 2); }

// A ROWS x BK block of an operand: global to registers, registers to [k][r].
template <int ROWS, int BK>
struct Block {
  static constexpr int kAll = ROWS * BK / 4, kVecs = kAll < kThreads ? 1 : kAll / kThreads;
  static_assert(kAll < kThreads || kVecs * kThreads == kAll, "whole vectors per thread");
  float4 v[kVecs];
  MOE_DEV void fetch(const Operand& o, int r0, int k0) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int t = threadIdx.x + i * kThreads;
      const int r = r0 + (o.ks == 1 ? t / (BK / 4) : t % (ROWS / 4) * 4);
      const int k = k0 + (o.ks == 1 ? t % (BK / 4) * 4 : t / (ROWS / 4));
      v[i] = t < kAll && r < o.rows && k < o.len ? *reinterpret_cast<const float4*>(o.p + r * o.rs + k * o.ks)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  MOE_DEV void put(float (&sm)[BK][ROWS], bool along_k) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int t = threadIdx.x + i * kThreads;
      if (t >= kAll) break;
      if (along_k) {
        const int r = t / (BK / 4), k = t % (BK / 4) * 4;
        sm[k][swz<ROWS>(k, r)] = v[i].x;
        sm[k + 1][swz<ROWS>(k, r)] = v[i].y;
        sm[k + 2][swz<ROWS>(k, r)] = v[i].z;
        sm[k + 3][swz<ROWS>(k, r)] = v[i].w;
      } else {
        const int r = t % (ROWS / 4) * 4, k = t / (ROWS / 4);
        *reinterpret_cast<float4*>(&sm[k][swz<ROWS>(k, r)]) = v[i];
      }
    }
  }
};

// What a thread has summed: the running chain (pairs of columns, for packed
// multiply-adds), and the chains before it, in registers or, for tiles whose
// chain takes 64 of them, in shared memory (each thread its own column).
template <int TM, int TN>
struct Sum {
  static constexpr bool kRegs = TM * TN <= 16;
  uint64_t c[TM][TN / 2] = {};
  float v[TM][TN];  // the result, after total()
  float t[kRegs ? TM : 1][kRegs ? TN : 1] = {};
  bool any = false;
  MOE_DEV void flush(float4 (*chains)[kThreads]) {
    total(chains);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; j += 4) {
        if constexpr (kRegs) {
          for (int q = 0; q < 4; ++q) t[i][j + q] = v[i][j + q];
        } else {
          chains[(i * TN + j) / 4][threadIdx.x] = make_float4(v[i][j], v[i][j + 1], v[i][j + 2], v[i][j + 3]);
        }
        c[i][j / 2] = c[i][j / 2 + 1] = 0;  // (0.0f, 0.0f)
      }
    any = true;
  }
  MOE_DEV void total(float4 (*chains)[kThreads]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; j += 4) {
        split_f32x2(c[i][j / 2], v[i][j], v[i][j + 1]);
        split_f32x2(c[i][j / 2 + 1], v[i][j + 2], v[i][j + 3]);
        if (!any) continue;
        float4 w;
        if constexpr (kRegs) w = make_float4(t[i][j], t[i][j + 1], t[i][j + 2], t[i][j + 3]);
        else w = chains[(i * TN + j) / 4][threadIdx.x];
        v[i][j] += w.x;
        v[i][j + 1] += w.y;
        v[i][j + 2] += w.z;
        v[i][j + 3] += w.w;
      }
  }
};

// c[i][..] += x[i] y[..], both read from shared memory in groups of four.
template <int TM, int TN, class X, class Y>
MOE_DEV void outer(uint64_t (&c)[TM][TN / 2], X x_at, Y y_at) {
  uint64_t y[TN / 2];
#pragma unroll
  for (int j = 0; j < TN; j += 4) {
    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(y_at(j));
    y[j / 2] = w.x;
    y[j / 2 + 1] = w.y;
  }
#pragma unroll
  for (int i = 0; i < TM; i += 4) {
    const float4 w = *reinterpret_cast<const float4*>(x_at(i));
    const float x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t xx = f32x2(x[q], x[q]);
#pragma unroll
      for (int j = 0; j < TN / 2; ++j) c[i + q][j] = fma_f32x2(xx, y[j], c[i + q][j]);
    }
  }
}

// Thread (tx, ty) of 16 x 16 holds rows 4 ty + 64 i + 0..3 and columns 4 tx + 64
// j + 0..3 of a BM x BN tile, in v[4 i + ..][4 j + ..].
template <int BM, int BN, int BK>
struct Tile {
  static constexpr int kTM = BM / 16, kTN = BN / 16;
  using Acc = Sum<kTM, kTN>;
  float a[2][BK][BM];
  float b[2][BK][BN];
  float4 chains[kTM * kTN <= 16 ? 1 : kTM * kTN / 4][kThreads];

  MOE_DEV static int row(int i) { return 4 * ((int)threadIdx.x >> 4) + 64 * (i / 4) + i % 4; }
  MOE_DEV static int col(int j) { return 4 * ((int)threadIdx.x & 15) + 64 * (j / 4) + j % 4; }

  // acc += the products over k < K; the next block's loads are in flight while
  // one is multiplied
  MOE_DEV void run(const Operand& A, int m0, const Operand& B, int n0, int K, Acc& acc) {
    if (K <= 0) return;
    Block<BM, BK> va;
    Block<BN, BK> vb;
    va.fetch(A, m0, 0);
    vb.fetch(B, n0, 0);
    __syncthreads();  // the buffers' last readers are done
    va.put(a[0], A.ks == 1);
    vb.put(b[0], B.ks == 1);
    int buf = 0;
    for (int k0 = 0; k0 < K; k0 += BK, buf ^= 1) {
      __syncthreads();
      const bool more = k0 + BK < K;
      if (more) {
        va.fetch(A, m0, k0 + BK);
        vb.fetch(B, n0, k0 + BK);
      }
#pragma unroll
      for (int kk = 0; kk < BK; ++kk)
        outer<kTM, kTN>(acc.c, [&](int i) { return &a[buf][kk][swz<BM>(kk, row(i))]; },
                        [&](int j) { return &b[buf][kk][swz<BN>(kk, col(j))]; });
      if (more) {
        va.put(a[buf ^ 1], A.ks == 1);
        vb.put(b[buf ^ 1], B.ks == 1);
      }
      if ((k0 + BK) % kChain == 0) acc.flush(chains);
    }
  }
  MOE_DEV void finish(Acc& acc) { acc.total(chains); }
};

// A tile of BM (8 or 32) x 32 for groups of few rows: kGroups groups of threads
// each take their part of every 64-deep block, so a tile's chain over k is as
// much shorter and a small product spreads over more threads. Such products wait
// for memory more than they compute, so two blocks are in flight (three
// spill: 32 rows of 256 x 512 matrices 78 instead of 70 us).
template <int BM>
struct SplitTile {
  static constexpr int kCols = 32, kBK = 64, kAhead = 2;
  static constexpr int kPart = BM / 4 * (kCols / 4), kGroups = kThreads / kPart;  // threads of a group, groups
  using Acc = Sum<4, 4>;
  union {
    struct {
      float a[2][kBK][BM];
      float b[2][kBK][kCols];
    };
    float sum[kGroups][BM][kCols];
  };
  // After finish(), thread t holds row t / 8 (none at or past BM), columns 4 (t % 8) + 0..3.
  MOE_DEV static int row() { return threadIdx.x / 8; }
  MOE_DEV static int col() { return threadIdx.x % 8 * 4; }

  MOE_DEV void run(const Operand& A, int m0, const Operand& B, int n0, int K, Acc& acc) {
    if (K <= 0) return;
    const int t = threadIdx.x % kPart, g = threadIdx.x / kPart, tx = t & 7, ty = t >> 3;
    Block<BM, kBK> va[kAhead];
    Block<kCols, kBK> vb[kAhead];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {  // (past K: zeros)
      va[s].fetch(A, m0, s * kBK);
      vb[s].fetch(B, n0, s * kBK);
    }
    __syncthreads();  // the buffers' last readers are done
    int buf = 0;
    for (int k1 = 0; k1 < K; k1 += kAhead * kBK) {
#pragma unroll
      for (int s = 0; s < kAhead; ++s, buf ^= 1) {
        const int k0 = k1 + s * kBK;
        if (k0 >= K) break;
        va[s].put(a[buf], A.ks == 1);
        vb[s].put(b[buf], B.ks == 1);
        if (k0 + kAhead * kBK < K) {
          va[s].fetch(A, m0, k0 + kAhead * kBK);
          vb[s].fetch(B, n0, k0 + kAhead * kBK);
        }
        __syncthreads();  // (the other buffer is read no longer, either)
#pragma unroll
        for (int q = 0; q < kBK / kGroups; ++q) {
          const int kk = g * (kBK / kGroups) + q;
          outer<4, 4>(acc.c, [&](int) { return &a[buf][kk][swz<BM>(kk, 4 * ty)]; },
                      [&](int) { return &b[buf][kk][swz<kCols>(kk, 4 * tx)]; });
        }
        if ((k0 / kBK + 1) % (kChain / (kBK / kGroups)) == 0) acc.flush(nullptr);
      }
    }
  }
  // The kGroups groups' sums, in order, as this thread's part of the tile.
  MOE_DEV void finish(Acc& acc, float (&out)[4]) {
    const int t = threadIdx.x % kPart, g = threadIdx.x / kPart, tx = t & 7, ty = t >> 3;
    acc.total(nullptr);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(&sum[g][4 * ty + i][4 * tx]) =
          make_float4(acc.v[i][0], acc.v[i][1], acc.v[i][2], acc.v[i][3]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = 0.f;
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      if (row() >= BM) break;
      const float4 v = *reinterpret_cast<const float4*>(&sum[q][row()][col()]);
      out[0] += v.x;
      out[1] += v.y;
      out[2] += v.z;
      out[3] += v.w;
    }
    __syncthreads();  // before the next unit's blocks
  }
};

}  // namespace simt
}  // namespace moe
