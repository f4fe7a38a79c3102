// Router backward: the gradient of the logits from the gradients of the
// gates, per token (one warp), and what joins the split weight gradient.
//
// With s the scores, S the selected experts, c = route_scale, Z = sum_S s:
//   normalised gates    ds_j = (c / Z) (dG_j - sum_S dG_i s_i / Z), j in S
//   otherwise           ds_j = c dG_j
//   sigmoid             dz_j = ds_j s_j (1 - s_j)
//   softmax             dz_j = s_j (ds_j - sum_S ds_i s_i)  (all experts; the
//                       sum is zero for normalised gates)
// The two products dx = dz W_r and dW_r = dz^T x run on the expert kernels.
// bf16 layers: dz is passed as two bf16 terms hi + lo (16 bits of mantissa),
// whose products are summed in fp32, so dz costs no visible rounding next to
// the bf16 W_r, x and results; fp32 layers use fp32 throughout.
#include <cfloat>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

MOE_DEV float wsum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
MOE_DEV float wmax(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// Lane l holds experts 32 j + l, j < V; slot i of the token sits in lane i.
template <int V>
__global__ void __launch_bounds__(256) route_dz_kernel(RouteDzArgs a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    // tables of the products: one group of T rows, and the row ranges of the
    // split weight gradient
    a.grp_row0[0] = 0;
    a.grp_rows[0] = (int32_t)a.T;
    a.grp_row0[1] = 0;
    a.grp_rows[1] = 0;
    a.unit_base[0] = 0;
    a.unit_base[1] = a.unit_base[2] = a.units;
    for (int i = 0; i < a.splits; ++i) {
      const int64_t lo = a.T * i / a.splits / 64 * 64, hi = i + 1 == a.splits ? a.T : a.T * (i + 1) / a.splits / 64 * 64;
      a.split_row0[i] = (int32_t)lo;
      a.split_rows[i] = (int32_t)(hi - lo);
    }
  }
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int N = a.N, k = a.k;
  float s[V], om[V], ds[V];  // scores, 1 - sigmoid, gradient of the scores
#pragma unroll
  for (int j = 0; j < V; ++j) {
    s[j] = 32 * j + lane < N ? a.logits[t * N + 32 * j + lane] : -INFINITY;
    om[j] = 1.f;
    ds[j] = 0.f;
  }
  if (a.score_fn == MOE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, s[j]);
    m = wmax(m);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j] = 32 * j + lane < N ? expf(s[j] - m) : 0.f;
      sum += s[j];
    }
    sum = wsum(sum);
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = s[j] / sum;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float z = s[j];
      s[j] = 32 * j + lane < N ? 1.f / (1.f + expf(-z)) : 0.f;
      om[j] = 1.f / (1.f + expf(z));
    }
  }
  // this lane's slot: its expert (-1: none), whether it is the expert's first
  // slot, and its rank among the token's distinct experts
  int e = -1;
  if (lane < k) {
    e = a.idx[t * k + lane];
    if (e < 0 || e >= N) {
      set_status(a.status, MOE_DEV_BAD_EXPERT);
      e = -1;
    }
  }
  bool firsts = e >= 0;
  for (int i = 0; i < k; ++i) {
    const int ei = __shfl_sync(0xffffffffu, e, i);
    if (i < lane && ei == e) firsts = false;
  }
  float dG = 0.f;
  if (a.slot_pos) {
    // the gradient of the slot's gate is that of the row the dispatch gave it:
    // slot_pos lists the token's rows by ascending expert
    int rank = 0;
    for (int i = 0; i < k; ++i) {
      const int ei = __shfl_sync(0xffffffffu, firsts ? e : -1, i);
      rank += ei >= 0 && ei < e;
    }
    if (firsts) {
      const int32_t row = a.slot_pos[t * k + rank];
      if (row >= 0 && row < a.T * k) dG = a.dgates[row];
    }
  } else if (e >= 0) {
    dG = a.dgates[t * k + lane];
  }
  float Z = 0.f, dot = 0.f, my_s = 0.f;
  for (int i = 0; i < k; ++i) {
    const int ei = __shfl_sync(0xffffffffu, e, i);
    if (ei < 0) continue;
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j == ei >> 5) v = s[j];
    v = __shfl_sync(0xffffffffu, v, ei & 31);
    Z += v;
    dot = fmaf(__shfl_sync(0xffffffffu, dG, i), v, dot);
    if (lane == i) my_s = v;
  }
  const float my_ds = a.normalize ? a.route_scale / Z * (dG - dot / Z) : a.route_scale * dG;
  for (int i = 0; i < k; ++i) {
    const int ei = __shfl_sync(0xffffffffu, e, i);
    const float v = __shfl_sync(0xffffffffu, my_ds, i);
    if (ei < 0 || lane != (ei & 31)) continue;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j == ei >> 5) ds[j] += v;
  }
  const float mean = a.score_fn == MOE_SOFTMAX && !a.normalize ? wsum(e >= 0 ? my_ds * my_s : 0.f) : 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = 32 * j + lane;
    if (col >= N) continue;
    const float dz = a.score_fn == MOE_SOFTMAX ? s[j] * (ds[j] - mean) : ds[j] * s[j] * om[j];
    if (a.dz) {
      a.dz[t * N + col] = dz;
    } else {
      const __nv_bfloat16 hi = __float2bfloat16_rn(dz);
      a.hi[t * a.ld + col] = hi;
      a.lo[t * a.ld + col] = __float2bfloat16_rn(dz - __bfloat162float(hi));
    }
  }
}

// dW = sum over the planes in order, rounded once (or added to an fp32 dW).
__global__ void __launch_bounds__(256) join_planes_kernel(const float4* __restrict__ planes, int n, int64_t vecs,
                                                          void* __restrict__ dW, int f32, int accumulate) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= vecs) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int q = 0; q < n; ++q) {
    const float4 w = __ldg(planes + q * vecs + i);
    v.x += w.x;
    v.y += w.y;
    v.z += w.z;
    v.w += w.w;
  }
  if (f32) {
    float4* o = static_cast<float4*>(dW) + i;
    if (accumulate) {
      const float4 w = *o;
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    *o = v;
  } else {
    static_cast<uint2*>(dW)[i] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

}  // namespace

cudaError_t launch_route_dz(const RouteDzArgs& a, cudaStream_t s) {
  const int warps = 8;
  const unsigned blocks = (unsigned)((a.T + warps - 1) / warps);
  const int V = (a.N + 31) / 32;
  if (V <= 1) route_dz_kernel<1><<<blocks, 32 * warps, 0, s>>>(a);
  else if (V <= 2) route_dz_kernel<2><<<blocks, 32 * warps, 0, s>>>(a);
  else if (V <= 4) route_dz_kernel<4><<<blocks, 32 * warps, 0, s>>>(a);
  else if (V <= 8) route_dz_kernel<8><<<blocks, 32 * warps, 0, s>>>(a);
  else route_dz_kernel<16><<<blocks, 32 * warps, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_join_planes(const float* planes, int n, int64_t elems, void* dW, int grad_dtype, bool accumulate,
                               cudaStream_t s) {
  const int64_t vecs = elems / 4;
  join_planes_kernel<<<(unsigned)((vecs + 255) / 256), 256, 0, s>>>(reinterpret_cast<const float4*>(planes), n, vecs,
                                                                    dW, grad_dtype == MOE_F32, accumulate);
  return cudaGetLastError();
}

}  // namespace moe
