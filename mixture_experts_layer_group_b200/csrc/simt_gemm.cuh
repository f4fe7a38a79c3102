// fp32 matrix products on CUDA cores: tiles of C[m, n] = sum_k A(m, k) B(n, k)
// with operands contiguous along either index, for the layers stored in fp32
// (tensor cores would round the operands to TF32). 256 threads.
//
// Each output is one chain of fused multiply-adds over ascending k, whatever
// the tile (SplitTile excepted: four chains, added in order), so a result does
// not depend on the tile that computed it.
#pragma once

#include "common.cuh"

namespace moe {
namespace simt {

constexpr int kThreads = 256;

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
MOE_DEV int swz(int k, int r) { return r ^ (((k >> 2) & 7) << 2); }

// A ROWS x BK block of an operand: global to registers, registers to [k][r].
template <int ROWS, int BK>
struct Block {
  static constexpr int kVecs = ROWS * BK / 4 / kThreads;
  static_assert(kVecs * kThreads * 4 == ROWS * BK, "whole vectors per thread");
  float4 v[kVecs];
  MOE_DEV void fetch(const Operand& o, int r0, int k0) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int t = threadIdx.x + i * kThreads;
      const int r = r0 + (o.ks == 1 ? t / (BK / 4) : t % (ROWS / 4) * 4);
      const int k = k0 + (o.ks == 1 ? t % (BK / 4) * 4 : t / (ROWS / 4));
      v[i] = r < o.rows && k < o.len ? __ldg(reinterpret_cast<const float4*>(o.p + r * o.rs + k * o.ks))
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  MOE_DEV void put(float (&sm)[BK][ROWS], bool along_k) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int t = threadIdx.x + i * kThreads;
      if (along_k) {
        const int r = t / (BK / 4), k = t % (BK / 4) * 4;
        sm[k][swz(k, r)] = v[i].x;
        sm[k + 1][swz(k, r)] = v[i].y;
        sm[k + 2][swz(k, r)] = v[i].z;
        sm[k + 3][swz(k, r)] = v[i].w;
      } else {
        const int r = t % (ROWS / 4) * 4, k = t / (ROWS / 4);
        *reinterpret_cast<float4*>(&sm[k][swz(k, r)]) = v[i];
      }
    }
  }
};

// Thread (tx, ty) of 16 x 16 holds rows 4 ty + 64 i + 0..3 and columns 4 tx + 64
// j + 0..3 of a BM x BN tile, in acc[4 i + ..][4 j + ..].
template <int BM, int BN, int BK>
struct Tile {
  static constexpr int kTM = BM / 16, kTN = BN / 16;
  float a[2][BK][BM];
  float b[2][BK][BN];

  MOE_DEV static int row(int i) { return 4 * ((int)threadIdx.x >> 4) + 64 * (i / 4) + i % 4; }
  MOE_DEV static int col(int j) { return 4 * ((int)threadIdx.x & 15) + 64 * (j / 4) + j % 4; }

  // acc += the products over k < K; the next block's loads are in flight while
  // one is multiplied
  MOE_DEV void run(const Operand& A, int m0, const Operand& B, int n0, int K, float (&acc)[kTM][kTN]) {
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
      for (int kk = 0; kk < BK; ++kk) {
        float x[kTM], y[kTN];
#pragma unroll
        for (int i = 0; i < kTM; i += 4)
          *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(&a[buf][kk][swz(kk, row(i))]);
#pragma unroll
        for (int j = 0; j < kTN; j += 4)
          *reinterpret_cast<float4*>(y + j) = *reinterpret_cast<const float4*>(&b[buf][kk][swz(kk, col(j))]);
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
          for (int j = 0; j < kTN; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
      }
      if (more) {
        va.put(a[buf ^ 1], A.ks == 1);
        vb.put(b[buf ^ 1], B.ks == 1);
      }
    }
  }
};

// A 32 x 32 tile for groups of few rows: four groups of 64 threads each take a
// quarter of every 64-deep block, so a tile's chain over k is four times
// shorter and a small product spreads over more threads.
struct SplitTile {
  static constexpr int kB = 32, kBK = 64, kGroups = 4;
  union {
    struct {
      float a[2][kBK][kB];
      float b[2][kBK][kB];
    };
    float sum[kGroups][kB][kB];
  };
  // After finish(), thread t holds row t / 8, columns 4 (t % 8) + 0..3.
  MOE_DEV static int row() { return threadIdx.x / 8; }
  MOE_DEV static int col() { return threadIdx.x % 8 * 4; }

  MOE_DEV void run(const Operand& A, int m0, const Operand& B, int n0, int K, float (&acc)[4][4]) {
    if (K <= 0) return;
    const int t = threadIdx.x & 63, g = threadIdx.x >> 6, tx = t & 7, ty = t >> 3;
    Block<kB, kBK> va, vb;
    va.fetch(A, m0, 0);
    vb.fetch(B, n0, 0);
    __syncthreads();
    va.put(a[0], A.ks == 1);
    vb.put(b[0], B.ks == 1);
    int buf = 0;
    for (int k0 = 0; k0 < K; k0 += kBK, buf ^= 1) {
      __syncthreads();
      const bool more = k0 + kBK < K;
      if (more) {
        va.fetch(A, m0, k0 + kBK);
        vb.fetch(B, n0, k0 + kBK);
      }
#pragma unroll
      for (int q = 0; q < kBK / kGroups; ++q) {
        const int kk = g * (kBK / kGroups) + q;
        float x[4], y[4];
        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(&a[buf][kk][swz(kk, 4 * ty)]);
        *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(&b[buf][kk][swz(kk, 4 * tx)]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
      }
      if (more) {
        va.put(a[buf ^ 1], A.ks == 1);
        vb.put(b[buf ^ 1], B.ks == 1);
      }
    }
  }
  // The four groups' sums, in order, as this thread's part of the tile.
  MOE_DEV void finish(const float (&acc)[4][4], float (&out)[4]) {
    const int t = threadIdx.x & 63, g = threadIdx.x >> 6, tx = t & 7, ty = t >> 3;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(&sum[g][4 * ty + i][4 * tx]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = 0.f;
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
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
