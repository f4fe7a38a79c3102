// Backward products of fp32 layers on CUDA cores (tensor cores would round
// the operands far beyond the fp32 tolerance): the grouped experts' three
// stages and the router's two products, as 64 x 64 tiles of
// C[m, n] = sum_k A(m, k) B(n, k) with fp32 accumulators.
//
//   dh     q = dy W2 per row, then per element (s = sigmoid(g), h = g s u)
//            dgate += q h, du = gate q g s, dg = gate q u s (1 + g (1 - s)),
//            gh = gate h
//   dx     dx = dg W1 + du W3
//   dW     dW1 = dg^T x, dW3 = du^T x, dW2 = dy^T gh over a group's rows
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kBM = kSimtBM, kBN = kSimtBN, kBK = 32;
constexpr int kThreads = 256;  // 16 x 16 threads, 4 x 4 outputs each
constexpr int kVecs = kBM * kBK / 4 / kThreads;  // 16-byte loads per thread, operand and K step
static_assert(kBM == kBN && kVecs * kThreads * 4 == kBM * kBK, "both operands load alike");

// A strided operand: element (r, k) at p[r * rs + k * ks] for r < rows and
// k < ks_len, zero elsewhere. One of the strides is 1, the other and the
// bound along the unit stride are multiples of 4, so four consecutive
// elements load as one aligned vector.
struct Operand {
  const float* p;
  int64_t rs, ks, rows, len;
};

// Two buffers of a 32 x 64 block of each operand, [k][r]. The 16-byte column
// groups of row k are permuted by k / 4, so that the four rows a k-contiguous
// vector is spread over, and the reads along a row, hit all banks.
struct Tile {
  float a[2][kBK][kBM];
  float b[2][kBK][kBN];
};
MOE_DEV int swz(int k, int r) { return r ^ (((k >> 2) & 7) << 2); }

MOE_DEV void fetch(const Operand& o, int64_t r0, int64_t k0, float4 (&v)[kVecs]) {
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int t = threadIdx.x + i * kThreads;
    const int64_t r = r0 + (o.ks == 1 ? t / (kBK / 4) : t % (kBM / 4) * 4);
    const int64_t k = k0 + (o.ks == 1 ? t % (kBK / 4) * 4 : t / (kBM / 4));
    v[i] = r < o.rows && k < o.len ? __ldg(reinterpret_cast<const float4*>(o.p + r * o.rs + k * o.ks))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}
MOE_DEV void put(float (&sm)[kBK][kBM], bool along_k, const float4 (&v)[kVecs]) {
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int t = threadIdx.x + i * kThreads;
    if (along_k) {
      const int r = t / (kBK / 4), k = t % (kBK / 4) * 4;
      sm[k][swz(k, r)] = v[i].x;
      sm[k + 1][swz(k, r)] = v[i].y;
      sm[k + 2][swz(k, r)] = v[i].z;
      sm[k + 3][swz(k, r)] = v[i].w;
    } else {
      const int r = t % (kBM / 4) * 4, k = t / (kBM / 4);
      *reinterpret_cast<float4*>(&sm[k][swz(k, r)]) = v[i];
    }
  }
}

// acc[i][j] += sum_{k < K} A(m0 + 4 ty + i, k) B(n0 + 4 tx + j, k). The next
// block's loads are in flight while a block is multiplied.
MOE_DEV void gemm_tile(Tile& sm, const Operand& A, int64_t m0, const Operand& B, int64_t n0, int64_t K,
                       float (&acc)[4][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (K <= 0) return;
  float4 va[kVecs], vb[kVecs];
  fetch(A, m0, 0, va);
  fetch(B, n0, 0, vb);
  __syncthreads();  // the buffers' last readers are done
  put(sm.a[0], A.ks == 1, va);
  put(sm.b[0], B.ks == 1, vb);
  int buf = 0;
  for (int64_t k0 = 0; k0 < K; k0 += kBK, buf ^= 1) {
    __syncthreads();
    const bool more = k0 + kBK < K;
    if (more) {
      fetch(A, m0, k0 + kBK, va);
      fetch(B, n0, k0 + kBK, vb);
    }
#pragma unroll
    for (int kk = 0; kk < kBK; ++kk) {
      const float4 a4 = *reinterpret_cast<const float4*>(&sm.a[buf][kk][swz(kk, 4 * ty)]);
      const float4 b4 = *reinterpret_cast<const float4*>(&sm.b[buf][kk][swz(kk, 4 * tx)]);
      const float a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    if (more) {
      put(sm.a[buf ^ 1], A.ks == 1, va);
      put(sm.b[buf ^ 1], B.ks == 1, vb);
    }
  }
}

struct Groups {
  const int32_t* unit_base;
  const int32_t* grp_row0;
  const int32_t* grp_rows;
  int N;
};

// Row-tile unit u -> its group, column tile and row tile (as the forward's).
MOE_DEV void find_unit(const Groups& gr, int u, int& g, int& f, int& m) {
  int lo = 0, hi = gr.N;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (gr.unit_base[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  g = lo;
  const int mt = (gr.grp_rows[g] + kBM - 1) / kBM;
  const int local = u - gr.unit_base[g];
  f = local / mt;
  m = local % mt;
}

struct DhParams {
  Groups gr;
  const float* dy;    // [R, d]
  const float* W2;    // [N, d, F]
  const float* gu;    // [R, 2 F]
  const float* gate;  // [R] or null
  float* dg;
  float* du;
  float* gh;
  float* part;        // [ceil(F / 64), R] or null
  int d, F;
  int64_t R;
};

__global__ void __launch_bounds__(kThreads) dh_simt_kernel(DhParams p) {
  __shared__ Tile sm;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int total = p.gr.unit_base[p.gr.N + 1];
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int g, f, m;
    find_unit(p.gr, u, g, f, m);
    const int rows = p.gr.grp_rows[g];
    const int64_t row0 = p.gr.grp_row0[g];
    float acc[4][4] = {};
    gemm_tile(sm, Operand{p.dy + row0 * p.d, p.d, 1, rows, p.d}, (int64_t)m * kBM,
              Operand{p.W2 + (int64_t)g * p.d * p.F, 1, p.F, p.F, p.d}, (int64_t)f * kBN, p.d, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = m * kBM + 4 * ty + i;
      const int64_t row = row0 + r;
      const bool in = r < rows;
      const float gate = in && p.gate ? p.gate[row] : 1.f;
      float dgate = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = f * kBN + 4 * tx + j;
        if (!in || c >= p.F) continue;
        const float gv = p.gu[row * 2 * p.F + c], uv = p.gu[row * 2 * p.F + p.F + c];
        const float s = 1.f / (1.f + expf(-gv)), a = gv * s, q = acc[i][j], dh = gate * q;
        dgate = fmaf(q, a * uv, dgate);
        p.du[row * p.F + c] = dh * a;
        p.dg[row * p.F + c] = dh * uv * s * (1.f + gv * (1.f - s));
        p.gh[row * p.F + c] = gate * a * uv;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) dgate += __shfl_xor_sync(0xffffffffu, dgate, off);
      if (p.part && in && tx == 0) p.part[(int64_t)f * p.R + row] = dgate;
    }
  }
}

struct DxParams {
  Groups gr;
  const float* d0;  // [R, F]: dg | dz (row stride ld)
  const float* d1;  // [R, F]: du | null
  const float* W0;  // [N, F, d]: W1 | W_r
  const float* W1;  // [N, F, d]: W3 | null
  float* dx;        // [R, d]
  int d, F;
  int64_t ld;       // a multiple of 4; columns F .. ld - 1 are zero
};

__global__ void __launch_bounds__(kThreads) dx_simt_kernel(DxParams p) {
  __shared__ Tile sm;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int total = p.gr.unit_base[p.gr.N + 1];
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int g, f, m;
    find_unit(p.gr, u, g, f, m);
    const int rows = p.gr.grp_rows[g];
    const int64_t row0 = p.gr.grp_row0[g], w0 = (int64_t)g * p.F * p.d;
    float acc[4][4] = {};
    gemm_tile(sm, Operand{p.d0 + row0 * p.ld, p.ld, 1, rows, p.ld}, (int64_t)m * kBM,
              Operand{p.W0 + w0, 1, p.d, p.d, p.F}, (int64_t)f * kBN, p.F, acc);
    if (p.d1)
      gemm_tile(sm, Operand{p.d1 + row0 * p.ld, p.ld, 1, rows, p.ld}, (int64_t)m * kBM,
                Operand{p.W1 + w0, 1, p.d, p.d, p.F}, (int64_t)f * kBN, p.F, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = m * kBM + 4 * ty + i;
      if (r >= rows) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = f * kBN + 4 * tx + j;
        if (c < p.d) p.dx[(row0 + r) * p.d + c] = acc[i][j];
      }
    }
  }
}

// dW[g][m][n] = sum over the rows r of group g of A[r][m] B[r][n].
struct DwMatrix {
  const float* A;  // [R, M], row stride lda (a multiple of 4; columns M .. lda - 1 are zero)
  const float* B;  // [R, N]
  float* out;      // [groups, M, N]
  int M, N;
  int64_t lda;
};
struct DwParams {
  DwMatrix mat[3];
  int nmat, groups;
  const int32_t* grp_row0;
  const int32_t* grp_rows;
  int accumulate;
};

__global__ void __launch_bounds__(kThreads) dw_simt_kernel(DwParams p, int64_t units) {
  __shared__ Tile sm;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    int64_t left = u;
    int i0 = 0;
    int64_t per = 0;
    for (;; ++i0) {
      per = (int64_t)((p.mat[i0].M + kBM - 1) / kBM) * ((p.mat[i0].N + kBN - 1) / kBN);
      if (i0 == p.nmat - 1 || left < per * p.groups) break;
      left -= per * p.groups;
    }
    const DwMatrix& x = p.mat[i0];
    const int g = (int)(left / per);
    const int64_t local = left % per;
    const int nt = (x.N + kBN - 1) / kBN;
    const int64_t m0 = local / nt * kBM, n0 = local % nt * kBN;
    const int64_t row0 = p.grp_row0[g];
    float acc[4][4] = {};
    const int rows = p.grp_rows[g];
    gemm_tile(sm, Operand{x.A + row0 * x.lda, 1, x.lda, x.lda, rows}, m0,
              Operand{x.B + row0 * x.N, 1, x.N, x.N, rows}, n0, rows, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + 4 * ty + i, n = n0 + 4 * tx + j;
        if (m >= x.M || n >= x.N) continue;
        float* o = x.out + ((int64_t)g * x.M + m) * x.N + n;
        *o = p.accumulate ? *o + acc[i][j] : acc[i][j];
      }
  }
}

int64_t dw_units(const DwParams& p) {
  int64_t n = 0;
  for (int i = 0; i < p.nmat; ++i)
    n += (int64_t)p.groups * ((p.mat[i].M + kBM - 1) / kBM) * ((p.mat[i].N + kBN - 1) / kBN);
  return n;
}

cudaError_t launch_dw(const DwParams& p, cudaStream_t s) {
  const int64_t units = dw_units(p), cap = (int64_t)device_sm_count() * 8;
  dw_simt_kernel<<<(unsigned)(units < cap ? units : cap), kThreads, 0, s>>>(p, units);
  return cudaGetLastError();
}

// 32 rows per CTA; warp w adds planes w, w + 8, ..., then the warps' sums are
// added in order (so that a row's planes are eight short chains of loads).
__global__ void __launch_bounds__(256) dgate_reduce_kernel(const float* __restrict__ part, int planes, int64_t rows,
                                                           float* __restrict__ dgate) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float sums[8][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (r < rows) {
#pragma unroll 8
    for (int i = w; i < planes; i += 8) v += __ldg(part + i * rows + r);
  }
  sums[w][lane] = v;
  __syncthreads();
  if (w || r >= rows) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) v += sums[i][lane];
  dgate[r] = v;
}

}  // namespace

cudaError_t launch_dgate_reduce(const float* part, int planes, int64_t rows, float* dgate, cudaStream_t s) {
  return launch_after(dgate_reduce_kernel, (unsigned)((rows + 31) / 32), 256, 0, s, part, planes, rows, dgate);
}

cudaError_t launch_experts_backward_simt(const Problem& p, const ExpertsBwdArgs& a, cudaStream_t s) {
  const int grid = device_sm_count() * 6;
  const Groups g1{a.unit_base1, a.grp_row0, a.grp_rows, p.N}, g2{a.unit_base2, a.grp_row0, a.grp_rows, p.N};
  DhParams h{g1, (const float*)a.dy_rows, (const float*)a.W2, (const float*)a.gu, a.gate_rows, (float*)a.dg,
             (float*)a.du, (float*)a.gh, a.dgate_rows ? a.dgate_part : nullptr, p.d, p.F, p.R};
  dh_simt_kernel<<<grid, kThreads, 0, s>>>(h);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.dgate_rows) e = launch_dgate_reduce(a.dgate_part, dgate_planes(p), p.R, a.dgate_rows, s);
  if (e == cudaSuccess && a.dx_rows) {
    DxParams x{g2, (const float*)a.dg, (const float*)a.du, (const float*)a.W1, (const float*)a.W3, (float*)a.dx_rows,
               p.d, p.F, p.F};
    dx_simt_kernel<<<grid, kThreads, 0, s>>>(x);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && a.dW1) {
    DwParams w{};
    w.mat[0] = {(const float*)a.dg, (const float*)a.x_rows, (float*)a.dW1, p.F, p.d, p.F};
    w.mat[1] = {(const float*)a.du, (const float*)a.x_rows, (float*)a.dW3, p.F, p.d, p.F};
    w.mat[2] = {(const float*)a.dy_rows, (const float*)a.gh, (float*)a.dW2, p.d, p.F, p.d};
    w.nmat = 3;
    w.groups = p.N;
    w.grp_row0 = a.grp_row0;
    w.grp_rows = a.grp_rows;
    w.accumulate = a.accumulate;
    e = launch_dw(w, s);
  }
  return e;
}

cudaError_t launch_route_products_simt(const Problem& p, const RouteBwdArgs& a, cudaStream_t s) {
  const int32_t* row0 = a.tables + kRtRow0;
  const int32_t* rows = a.tables + kRtRows;
  cudaError_t e = cudaSuccess;
  if (a.dx) {
    DxParams x{Groups{a.tables + kRtUnits, row0, rows, 1}, a.dz, nullptr, (const float*)a.W_r, nullptr,
               (float*)a.dx, p.d, p.N, a.ld};
    dx_simt_kernel<<<device_sm_count() * 6, kThreads, 0, s>>>(x);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && a.dW_r) {
    DwParams w{};
    w.mat[0] = {a.dz, (const float*)a.x, (float*)a.dW_r, p.N, p.d, a.ld};
    w.nmat = 1;
    w.groups = 1;
    w.grp_row0 = row0;
    w.grp_rows = rows;
    w.accumulate = a.accumulate;
    e = launch_dw(w, s);
  }
  return e;
}

}  // namespace moe
