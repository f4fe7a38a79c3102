// The training forward and backward of fp32 layers on CUDA cores: the grouped
// experts' products and the router's two, with fp32 accumulators.
//
//   gu     g = x W1^T, u = x W3^T; then h = silu(g) u and y = gate (h W2^T)
//   dh     q = dy W2 per row, then per element (s = sigmoid(g), h = g s u)
//            dgate += q h, du = gate q g s, dg = gate q u s (1 + g (1 - s)),
//            gh = gate h
//   dx     dx = dg W1 + du W3
//   dW     dW1 = dg^T x, dW3 = du^T x, dW2 = dy^T gh over a group's rows
//
// Bound by the FP32 pipes where the rows are many: 8 groups of 512 rows, d 1024,
// d_ff 1024 take 661 us forward (25.8 GFLOP, 39 TFLOP/s) and 1290 us backward in
// tiles of 128 x 128 (8 x 8 outputs per thread, four 16-byte shared loads for 32
// packed multiply-adds of two; unpacked ones 704 and 1420 us). Few rows leave SMs
// idle and make long chains of dependent blocks, so small products take tiles
// of 32 x 32 or 8 x 32 whose sum is split over groups of threads: 16 groups of 32
// rows, d 256, d_ff 512 take 46 us forward and 67 us backward (0.8 GFLOP); one
// group of 3 rows of 7168 x 4096 takes 137 us forward (352 MB of weights, 2.6
// TB/s). The weight gradients run beside the dx product, which like them needs
// only dh (15 us of the smaller backward).
#include <cmath>
#include <type_traits>

#include "internal.h"
#include "simt_gemm.cuh"

namespace moe {
namespace {

using simt::kThreads;
using simt::Operand;
using simt::SplitTile;
using BigTile = simt::Tile<128, 128, 16>;
using MidTile = simt::Tile<64, 64, 32>;
// Tiles by their rows: 128, 64, or split ones of 32 or 8 rows and 32 columns.
__host__ __device__ constexpr bool is_split(int rows) { return rows <= 32; }
template <int B>
using TileOf = std::conditional_t<B == 128, BigTile, std::conditional_t<B == 64, MidTile, SplitTile<B < 32 ? 8 : 32>>>;

template <class T>
MOE_DEV T& tile_smem() {
  extern __shared__ float4 simt_smem[];
  return *reinterpret_cast<T*>(simt_smem);
}
template <class T, class... Params, class... Args>
cudaError_t launch_tile(void (*kernel)(Params...), unsigned blocks, cudaStream_t s, const Args&... args) {
  if (sizeof(T) > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(T));
    if (e != cudaSuccess) return e;
  }
  return launch_after(kernel, blocks, kThreads, sizeof(T), s, args...);
}

struct Groups {
  const int32_t* unit_base;
  const int32_t* grp_row0;
  const int32_t* grp_rows;
  int N;
};

// Row-tile unit u -> its group, column tile and row tile (as the forward's).
MOE_DEV void find_unit(const Groups& gr, int bm, int u, int& g, int& f, int& m) {
  int lo = 0, hi = gr.N;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (gr.unit_base[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  g = lo;
  const int mt = (gr.grp_rows[g] + bm - 1) / bm;
  const int local = u - gr.unit_base[g];
  f = local / mt;
  m = local - f * mt;
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
  float* part;        // [dgate_planes, R] or null
  int d, F;
  int64_t R;
};

// Four neighbouring features c .. c + 3 (all in or all out: F is a multiple of
// 8) of one row from q; returns their part of the gate's gradient.
MOE_DEV float dh_quad(const DhParams& p, int64_t row, int c, const float* q, float gate) {
  if (c >= p.F) return 0.f;
  const float4 g4 = __ldg(reinterpret_cast<const float4*>(p.gu + row * 2 * p.F + c));
  const float4 u4 = __ldg(reinterpret_cast<const float4*>(p.gu + row * 2 * p.F + p.F + c));
  const float g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
  float dg[4], du[4], gh[4], dgate = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float s = 1.f / (1.f + expf(-g[j])), a = g[j] * s, dh = gate * q[j];
    dgate = fmaf(q[j], a * u[j], dgate);
    du[j] = dh * a;
    dg[j] = dh * u[j] * s * (1.f + g[j] * (1.f - s));
    gh[j] = gate * a * u[j];
  }
  const int64_t at = row * p.F + c;
  *reinterpret_cast<float4*>(p.dg + at) = make_float4(dg[0], dg[1], dg[2], dg[3]);
  *reinterpret_cast<float4*>(p.du + at) = make_float4(du[0], du[1], du[2], du[3]);
  *reinterpret_cast<float4*>(p.gh + at) = make_float4(gh[0], gh[1], gh[2], gh[3]);
  return dgate;
}

template <int kB>
__global__ void __launch_bounds__(kThreads, 2) dh_simt_kernel(DhParams p) {
  using T = TileOf<kB>;
  constexpr int kBN = simt_cols(kB);
  T& sm = tile_smem<T>();
  griddep_launch_dependents();
  griddep_wait();
  const int total = p.gr.unit_base[p.gr.N + 1];
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int g, f, m;
    find_unit(p.gr, kB, u, g, f, m);
    const int rows = p.gr.grp_rows[g];
    const int64_t row0 = p.gr.grp_row0[g];
    const Operand A{p.dy + row0 * p.d, p.d, 1, rows, p.d}, B{p.W2 + (int64_t)g * p.d * p.F, 1, p.F, p.F, p.d};
    float* part = p.part ? p.part + (int64_t)f * p.R + row0 : nullptr;
    if constexpr (!is_split(kB)) {
      typename T::Acc acc;
      sm.run(A, m * kB, B, f * kBN, p.d, acc);
      sm.finish(acc);
#pragma unroll
      for (int i = 0; i < T::kTM; ++i) {
        const int r = m * kB + T::row(i);
        const bool in = r < rows;
        const float gate = in && p.gate ? p.gate[row0 + r] : 1.f;
        float dgate = 0.f;
        if (in)
#pragma unroll
          for (int j = 0; j < T::kTN; j += 4)
            dgate += dh_quad(p, row0 + r, f * kBN + T::col(j), &acc.v[i][j], gate);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) dgate += __shfl_xor_sync(0xffffffffu, dgate, off);
        if (part && in && (threadIdx.x & 15) == 0) part[r] = dgate;
      }
    } else {
      typename T::Acc acc;
      float q[4];
      sm.run(A, m * kB, B, f * kBN, p.d, acc);
      sm.finish(acc, q);
      const int r = m * kB + T::row();
      const bool in = T::row() < kB && r < rows;
      const float gate = in && p.gate ? p.gate[row0 + r] : 1.f;
      float dgate = in ? dh_quad(p, row0 + r, f * kBN + T::col(), q, gate) : 0.f;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) dgate += __shfl_xor_sync(0xffffffffu, dgate, off);
      if (part && in && (threadIdx.x & 7) == 0) part[r] = dgate;
    }
  }
}

// out[r][c] = gate_r sum_k A[r][k] B[c][k]: g and u of the training forward (B = W1
// and W3, halves of gu), and its down product.
struct FwdParams {
  Groups gr;
  const float* A;    // [R, K]
  const float* B0;   // [N, cols, K]
  const float* B1;   // a second such matrix, or null
  const float* gate; // [R] or null
  float* out;        // [R, cols], or [R, 2 cols]
  int K, cols;
};

template <int kB>
__global__ void __launch_bounds__(kThreads, 2) fwd_simt_kernel(FwdParams p) {
  using T = TileOf<kB>;
  constexpr int kBN = simt_cols(kB);
  T& sm = tile_smem<T>();
  griddep_launch_dependents();
  griddep_wait();
  const int mats = p.B1 ? 2 : 1, total = p.gr.unit_base[p.gr.N + 1] * mats;
  const int64_t ldo = (int64_t)p.cols * mats;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int g, f, m;
    find_unit(p.gr, kB, u / mats, g, f, m);
    const int which = u % mats, rows = p.gr.grp_rows[g];
    const int64_t row0 = p.gr.grp_row0[g];
    const float* B = (which ? p.B1 : p.B0) + (int64_t)g * p.cols * p.K;
    typename T::Acc acc;
    sm.run(Operand{p.A + row0 * p.K, p.K, 1, rows, p.K}, m * kB, Operand{B, p.K, 1, p.cols, p.K}, f * kBN, p.K, acc);
    auto put = [&](int r, int c, const float* v) {  // four columns (their number is a multiple of 8)
      if (r >= rows || c >= p.cols) return;
      const float gate = p.gate ? p.gate[row0 + r] : 1.f;
      *reinterpret_cast<float4*>(p.out + (row0 + r) * ldo + which * p.cols + c) =
          make_float4(gate * v[0], gate * v[1], gate * v[2], gate * v[3]);
    };
    if constexpr (!is_split(kB)) {
      sm.finish(acc);
#pragma unroll
      for (int i = 0; i < T::kTM; ++i)
#pragma unroll
        for (int j = 0; j < T::kTN; j += 4) put(m * kB + T::row(i), f * kBN + T::col(j), &acc.v[i][j]);
    } else {
      float v[4];
      sm.finish(acc, v);
      if (T::row() < kB) put(m * kB + T::row(), f * kBN + T::col(), v);
    }
  }
}

// h = silu(g) u, four features per thread.
__global__ void __launch_bounds__(256) swiglu_kernel(const float* gu, int F, int64_t vecs, float* h) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= vecs) return;
  const int64_t r = i / (F / 4), c = i % (F / 4) * 4;
  const float4 g = *reinterpret_cast<const float4*>(gu + r * 2 * F + c);
  const float4 u = *reinterpret_cast<const float4*>(gu + r * 2 * F + F + c);
  auto act = [](float a, float b) { return a / (1.f + expf(-a)) * b; };
  *reinterpret_cast<float4*>(h + r * F + c) = make_float4(act(g.x, u.x), act(g.y, u.y), act(g.z, u.z), act(g.w, u.w));
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
  int* publish;     // the flag of publish_waited(), or null
};

template <int kB>
__global__ void __launch_bounds__(kThreads, 2) dx_simt_kernel(DxParams p) {
  using T = TileOf<kB>;
  constexpr int kBN = simt_cols(kB);
  T& sm = tile_smem<T>();
  griddep_wait();
  if (threadIdx.x == 0) {  // (only now: the weight gradients read what dx waited for)
    if (p.publish && blockIdx.x == 0) publish_waited(p.publish);
    griddep_launch_dependents();
  }
  const int total = p.gr.unit_base[p.gr.N + 1];
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int g, f, m;
    find_unit(p.gr, kB, u, g, f, m);
    const int rows = p.gr.grp_rows[g];
    const int64_t row0 = p.gr.grp_row0[g], w0 = (int64_t)g * p.F * p.d;
    typename T::Acc acc;
    sm.run(Operand{p.d0 + row0 * p.ld, p.ld, 1, rows, (int)p.ld}, m * kB, Operand{p.W0 + w0, 1, p.d, p.d, p.F}, f * kBN,
           p.F, acc);
    if (p.d1)
      sm.run(Operand{p.d1 + row0 * p.ld, p.ld, 1, rows, (int)p.ld}, m * kB, Operand{p.W1 + w0, 1, p.d, p.d, p.F},
             f * kBN, p.F, acc);
    auto put = [&](int r, int c, const float* v) {  // four columns (d is a multiple of 8)
      if (r < rows && c < p.d)
        *reinterpret_cast<float4*>(p.dx + (row0 + r) * p.d + c) = make_float4(v[0], v[1], v[2], v[3]);
    };
    if constexpr (!is_split(kB)) {
      sm.finish(acc);
#pragma unroll
      for (int i = 0; i < T::kTM; ++i)
#pragma unroll
        for (int j = 0; j < T::kTN; j += 4) put(m * kB + T::row(i), f * kBN + T::col(j), &acc.v[i][j]);
    } else {
      float v[4];
      sm.finish(acc, v);
      if (T::row() < kB) put(m * kB + T::row(), f * kBN + T::col(), v);
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
  int per_group[3];  // tiles of a group's matrix
  const int32_t* grp_row0;
  const int32_t* grp_rows;
  int accumulate;
  const int* ready;  // null, or the predecessor's flag: it has waited for what this reads, which runs beside it
  unsigned* status;
};

template <class T, int kB>
__global__ void __launch_bounds__(kThreads, 2) dw_simt_kernel(DwParams p, int units) {
  T& sm = tile_smem<T>();
  griddep_launch_dependents();
  if (p.ready) {
    const bool go = threadIdx.x > 0 || take_published(p.ready);
    if (!go) set_status(p.status, MOE_DEV_WAIT_TIMEOUT);
    if (!__syncthreads_and(go)) units = 0;
  } else {
    griddep_wait();
  }
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    int i0 = 0, left = u;
    while (i0 < p.nmat - 1 && left >= p.per_group[i0] * p.groups) left -= p.per_group[i0++] * p.groups;
    const DwMatrix& x = p.mat[i0];
    const int g = left / p.per_group[i0], local = left - g * p.per_group[i0];
    const int nt = (x.N + kB - 1) / kB, mi = local / nt;
    const int m0 = mi * kB, n0 = (local - mi * nt) * kB;
    const int64_t row0 = p.grp_row0[g];
    const int rows = p.grp_rows[g];
    typename T::Acc acc;
    sm.run(Operand{x.A + row0 * x.lda, 1, x.lda, (int)x.lda, rows}, m0, Operand{x.B + row0 * x.N, 1, x.N, x.N, rows}, n0,
           rows, acc);
    sm.finish(acc);
#pragma unroll
    for (int i = 0; i < T::kTM; ++i)
#pragma unroll
      for (int j = 0; j < T::kTN; j += 4) {
        const int m = m0 + T::row(i), n = n0 + T::col(j);
        if (m >= x.M || n >= x.N) continue;  // N is a multiple of 8: four columns are in or out
        float4* o = reinterpret_cast<float4*>(x.out + ((int64_t)g * x.M + m) * x.N + n);
        float4 v = make_float4(acc.v[i][j], acc.v[i][j + 1], acc.v[i][j + 2], acc.v[i][j + 3]);
        if (p.accumulate) {
          const float4 w = *o;
          v = make_float4(w.x + v.x, w.y + v.y, w.z + v.z, w.w + v.w);
        }
        *o = v;
      }
  }
  if (p.ready) griddep_wait();  // this grid ends after its predecessor
}

template <class T, int kB>
cudaError_t launch_dw_tile(DwParams p, cudaStream_t s) {
  int64_t units = 0;
  for (int i = 0; i < p.nmat; ++i) {
    const int64_t n = (int64_t)((p.mat[i].M + kB - 1) / kB) * ((p.mat[i].N + kB - 1) / kB);
    units += n * p.groups;
    p.per_group[i] = (int)n;
  }
  if (units > (1ll << 30)) return cudaErrorInvalidValue;
  const int64_t cap = (int64_t)device_sm_count() * 4;
  return launch_tile<T>(dw_simt_kernel<T, kB>, (unsigned)(units < cap ? units : cap), s, p, (int)units);
}

// Tiles of 128 where they fill the GPU, of 64 otherwise. The whole backward with
// 64 against 128: 8 groups, d 1024, d_ff 1024 (1536 tiles of 128) of 512 rows
// 1539 and 1390 us, of 16 rows 171 and 148 us. The router's few tiles (16 of
// them at 64 experts, d 1024, 4096 tokens) took 242 and 529 us without a split.
cudaError_t launch_dw(const DwParams& p, cudaStream_t s) {
  int64_t big = 0;
  for (int i = 0; i < p.nmat; ++i) big += (int64_t)(p.mat[i].M / 128) * (p.mat[i].N / 128) * p.groups;
  return big >= 2 * device_sm_count() ? launch_dw_tile<BigTile, 128>(p, s) : launch_dw_tile<MidTile, 64>(p, s);
}

// 32 rows per CTA; warp w adds planes w, w + 8, ..., then the warps' sums are
// added in order (so that a row's planes are eight short chains of loads).
__global__ void __launch_bounds__(256) dgate_reduce_kernel(const float* part, int planes, int64_t rows, const int32_t* units,
                                                           float* dgate) {
  griddep_launch_dependents();
  griddep_wait();
  if (*units == 0) return;  // counts that do not add up: no row was computed
  __shared__ float sums[8][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (r < rows) {
#pragma unroll 8
    for (int i = w; i < planes; i += 8) v += part[i * rows + r];
  }
  sums[w][lane] = v;
  __syncthreads();
  if (w || r >= rows) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) v += sums[i][lane];
  dgate[r] = v;
}

}  // namespace

cudaError_t launch_dgate_reduce(const float* part, int planes, int64_t rows, const int32_t* units, float* dgate,
                                cudaStream_t s) {
  return launch_after(dgate_reduce_kernel, (unsigned)((rows + 31) / 32), 256, 0, s, part, planes, rows, units, dgate);
}

// The row products' tiles, by the columns of their outputs: larger ones where the
// products give every SM two of 128 or four of 64. The whole backward (dx before
// the weight gradients, not beside them) with tiles of 128, 64 and 32 rows: 8
// groups of 512 rows (d 1024, d_ff 1024) 1390, 1510 and 1680 us, of 128 rows
// 669, 552 and 484 us; 16 groups of 256 rows (d 256, d_ff 512) 361, 257 and 290
// us, of 32 rows 234, 111 and 85 us. One group of 3 rows (d 7168, d_ff 4096)
// with tiles of 32 and 8 rows: 462 and 314 us.
int simt_tile(const Problem& p, int64_t cols) {
  const int64_t sms = device_sm_count();
  if ((p.R + 127) / 128 * (cols / 128) >= 2 * sms) return 128;
  if ((p.R + 63) / 64 * (cols / 64) >= 4 * sms) return 64;
  return p.R <= 8 * (int64_t)p.N ? 8 : 32;
}
int simt_train_tile(const Problem& p) { return simt_tile(p, 2 * (int64_t)p.F + p.d); }
int simt_bwd_tile(const Problem& p) { return simt_tile(p, (int64_t)p.F + p.d); }

cudaError_t launch_dh(const DhParams& h, int tile, cudaStream_t s) {
  const unsigned sms = device_sm_count();
  if (tile == 128) return launch_tile<TileOf<128>>(dh_simt_kernel<128>, sms * 2, s, h);
  if (tile == 64) return launch_tile<TileOf<64>>(dh_simt_kernel<64>, sms * 4, s, h);
  if (tile == 32) return launch_tile<TileOf<32>>(dh_simt_kernel<32>, sms * 6, s, h);
  return launch_tile<TileOf<8>>(dh_simt_kernel<8>, sms * 6, s, h);
}
cudaError_t launch_dx(const DxParams& x, int tile, cudaStream_t s) {
  const unsigned sms = device_sm_count();
  if (tile == 128) return launch_tile<TileOf<128>>(dx_simt_kernel<128>, sms * 2, s, x);
  if (tile == 64) return launch_tile<TileOf<64>>(dx_simt_kernel<64>, sms * 4, s, x);
  if (tile == 32) return launch_tile<TileOf<32>>(dx_simt_kernel<32>, sms * 6, s, x);
  return launch_tile<TileOf<8>>(dx_simt_kernel<8>, sms * 6, s, x);
}

cudaError_t launch_fwd(const FwdParams& f, int tile, cudaStream_t s) {
  const unsigned sms = device_sm_count();
  if (tile == 128) return launch_tile<TileOf<128>>(fwd_simt_kernel<128>, sms * 2, s, f);
  if (tile == 64) return launch_tile<TileOf<64>>(fwd_simt_kernel<64>, sms * 4, s, f);
  if (tile == 32) return launch_tile<TileOf<32>>(fwd_simt_kernel<32>, sms * 6, s, f);
  return launch_tile<TileOf<8>>(fwd_simt_kernel<8>, sms * 6, s, f);
}

cudaError_t launch_experts_train_simt(const Problem& p, const GemmArgs& a, cudaStream_t s) {
  const int tile = simt_train_tile(p);
  const Groups g1{a.unit_base1, a.grp_row0, a.grp_rows, p.N}, g2{a.unit_base2, a.grp_row0, a.grp_rows, p.N};
  cudaError_t e = launch_fwd(FwdParams{g1, (const float*)a.x_perm, (const float*)a.W1, (const float*)a.W3, nullptr,
                                       (float*)a.gu, p.d, p.F}, tile, s);
  const int64_t vecs = p.R * (int64_t)(p.F / 4);
  if (e == cudaSuccess)
    e = launch_after(swiglu_kernel, (unsigned)((vecs + 255) / 256), 256, 0, s, (const float*)a.gu, p.F, vecs,
                     (float*)a.h_perm);
  if (e != cudaSuccess) return e;
  return launch_fwd(FwdParams{g2, (const float*)a.h_perm, (const float*)a.W2, nullptr, a.gate_perm,
                              (float*)a.y_rows, p.F, p.d}, tile, s);
}

cudaError_t launch_experts_backward_simt(const Problem& p, const ExpertsBwdArgs& a, cudaStream_t s) {
  const int tile = simt_bwd_tile(p);
  const Groups g1{a.unit_base1, a.grp_row0, a.grp_rows, p.N}, g2{a.unit_base2, a.grp_row0, a.grp_rows, p.N};
  DhParams h{g1, (const float*)a.dy_rows, (const float*)a.W2, (const float*)a.gu, a.gate_rows, (float*)a.dg,
             (float*)a.du, (float*)a.gh, a.dgate_rows ? a.dgate_part : nullptr, p.d, p.F, p.R};
  cudaError_t e = launch_dh(h, tile, s);
  if (e == cudaSuccess && a.dx_rows) {
    DxParams x{g2, (const float*)a.dg, (const float*)a.du, (const float*)a.W1, (const float*)a.W3, (float*)a.dx_rows,
               p.d, p.F, p.F, a.dW1 ? a.sched + kSchedReady : nullptr};
    e = launch_dx(x, tile, s);
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
    w.ready = a.dx_rows ? a.sched + kSchedReady : nullptr;
    w.status = a.status;
    e = launch_dw(w, s);
  }
  if (e == cudaSuccess && a.dgate_rows)
    e = launch_dgate_reduce(a.dgate_part, dgate_planes(p), p.R, a.unit_base1 + p.N + 1, a.dgate_rows, s);
  return e;
}

cudaError_t launch_route_products_simt(const Problem& p, const RouteBwdArgs& a, cudaStream_t s) {
  const int32_t* row0 = a.tables + kRtRow0;
  const int32_t* rows = a.tables + kRtRows;
  Problem one = p;  // one group of T rows
  one.F = p.d;
  one.N = 1;
  one.R = p.T;
  cudaError_t e = cudaSuccess;
  if (a.dx) {
    DxParams x{Groups{a.tables + kRtUnits, row0, rows, 1}, a.dz, nullptr, (const float*)a.W_r, nullptr,
               (float*)a.dx, p.d, p.N, a.ld, a.dW_r ? a.tables + kRtReady : nullptr};
    e = launch_dx(x, simt_bwd_tile(one), s);
  }
  if (e == cudaSuccess && a.dW_r) {
    const bool split = a.splits > 1;
    DwParams w{};
    w.mat[0] = {a.dz, (const float*)a.x, split ? a.planes : (float*)a.dW_r, p.N, p.d, a.ld};
    w.nmat = 1;
    w.groups = a.splits;
    w.grp_row0 = a.tables + kRtSplit0;
    w.grp_rows = a.tables + kRtSplitRows;
    w.accumulate = !split && a.accumulate;
    w.ready = a.dx ? a.tables + kRtReady : nullptr;
    w.status = a.status;
    e = launch_dw_tile<MidTile, 64>(w, s);
    if (e == cudaSuccess && split)
      e = launch_join_planes(a.planes, a.splits, (int64_t)p.N * p.d, a.dW_r, a.grad_dtype, a.accumulate, s);
  }
  return e;
}

}  // namespace moe
