// Router backward: the gradient of the logits from the gradients of the
// gates, per token (one warp), and what joins the split weight gradient.
//
// With s the scores, S the selected experts, c = route_scale, Z = sum_S s:
//   normalised gates    ds_j = (c / Z) (dG_j - sum_S dG_i s_i / Z), j in S
//   otherwise           ds_j = c dG_j
//   sigmoid             dz_j = ds_j s_j (1 - s_j)
//   softmax             dz_j = s_j (ds_j - sum_S ds_i s_i)  (all experts; the
//                       sum is zero for normalised gates)
// The two products dx = dz W_r and dW_r = dz^T x then run as sums over rows:
// of dz^T and W_r (the experts), and of dz and x (the tokens). bf16 layers
// round dz to bf16 for them, as the experts' dg and du are (one rounding per
// term of sums kept in fp32); dz is written both ways. fp32 layers keep fp32.
//
// The kernel reads the logits once and writes dz twice (2 T N of each): a few
// microseconds at any size here, next to the products.
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

constexpr int kDzTokens = 16;  // tokens of a CTA: 32-byte runs of the transposed dz
constexpr int kDzWarps = 16;

// One warp per token. Lane l holds experts 32 j + l, j < V; slot
// i of the token sits in lane i.
template <int V>
__global__ void __launch_bounds__(32 * kDzWarps) route_dz_kernel(const __grid_constant__ RouteDzArgs a) {
  griddep_launch_dependents();
  __shared__ __nv_bfloat16 tile[32 * V][kDzTokens + 2];  // [expert][token] (+2: rows start in different banks)
  if (blockIdx.x == 0 && threadIdx.x < kRouteTables) a.tables[threadIdx.x] = a.table_values[threadIdx.x];
  const int lane = threadIdx.x & 31;
  const int N = a.N, k = a.k;
  const int64_t t0 = (int64_t)blockIdx.x * kDzTokens;
  for (int w = threadIdx.x >> 5; w < kDzTokens; w += kDzWarps) {
    const int64_t t = t0 + w;
    if (t >= a.T) break;
    float s[V], om[V], ds[V];  // scores, 1 - sigmoid, gradient of the scores
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j] = 32 * j + lane < N ? __ldg(a.logits + t * N + 32 * j + lane) : -INFINITY;
      om[j] = 1.f;
      ds[j] = 0.f;
    }
    // this lane's slot: its expert (-1: none) and logit, and whether it is the expert's first slot
    int e = lane < k ? __ldg(a.idx + t * k + lane) : -1;
    if (lane < k && (e < 0 || e >= N)) {
      set_status(a.status, MOE_DEV_BAD_EXPERT);
      e = -1;
    }
    float my_s = e >= 0 ? __ldg(a.logits + t * N + e) : -INFINITY;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const bool firsts = e >= 0 && lane == __ffs(same) - 1;
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
        const int32_t row = __ldg(a.slot_pos + t * k + rank);
        if (row >= 0 && row < a.T * k) dG = __ldg(a.dgates + row);
      }
    } else if (e >= 0) {
      dG = __ldg(a.dgates + t * k + lane);
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
      const float inv = 1.f / wsum(sum);
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] *= inv;
      my_s = e >= 0 ? expf(my_s - m) * inv : 0.f;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float z = s[j];
        s[j] = 32 * j + lane < N ? 1.f / (1.f + expf(-z)) : 0.f;
        om[j] = 1.f / (1.f + expf(z));  // 1 - s without its cancellation
      }
      my_s = e >= 0 ? 1.f / (1.f + expf(-my_s)) : 0.f;
    }
    float my_ds = a.route_scale * dG;
    float mean = 0.f;  // sum of ds_i s_i over the slots (zero for normalised gates)
    if (a.normalize) {
      const float Z = wsum(my_s), dot = wsum(dG * my_s);
      my_ds = a.route_scale / Z * (dG - dot / Z);
    } else if (a.score_fn == MOE_SOFTMAX) {
      mean = wsum(my_ds * my_s);
    }
    for (int i = 0; i < k; ++i) {
      const int ei = __shfl_sync(0xffffffffu, e, i);
      const float v = __shfl_sync(0xffffffffu, my_ds, i);
      if (ei < 0 || lane != (ei & 31)) continue;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j == ei >> 5) ds[j] += v;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = 32 * j + lane;
      const float dz = a.score_fn == MOE_SOFTMAX ? s[j] * (ds[j] - mean) : ds[j] * s[j] * om[j];
      if (a.dz) {
        // (columns N .. ld - 1 are zero)
        if (col < a.ld) a.dz[t * a.ld + col] = col < N ? dz : 0.f;
      } else if (col < N) {
        const __nv_bfloat16 v = __float2bfloat16_rn(dz);
        a.dz16[t * a.ld + col] = v;
        tile[col][w] = v;
      }
    }
  }
  if (a.dz || !a.dz16_t) return;
  __syncthreads();
  for (int i = threadIdx.x; i < N * (kDzTokens / 2); i += blockDim.x) {
    const int n = i / (kDzTokens / 2), c = i % (kDzTokens / 2) * 2;
    // a pair that starts inside T may end one past it, in the row's padding
    if (t0 + c < a.T)
      *reinterpret_cast<uint32_t*>(a.dz16_t + (int64_t)n * a.ld_t + t0 + c) =
          *reinterpret_cast<const uint32_t*>(&tile[n][c]);
  }
}

// dW = sum over the planes in order, rounded once (or added to an fp32 dW).
__global__ void __launch_bounds__(256) join_planes_kernel(const float4* __restrict__ planes, int n, int64_t vecs,
                                                          void* __restrict__ dW, int f32, int accumulate) {
  griddep_wait();
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
  const unsigned blocks = (unsigned)((a.T + kDzTokens - 1) / kDzTokens);
  const int V = (a.N + 31) / 32, threads = 32 * kDzWarps;
  if (V <= 1) route_dz_kernel<1><<<blocks, threads, 0, s>>>(a);
  else if (V <= 2) route_dz_kernel<2><<<blocks, threads, 0, s>>>(a);
  else if (V <= 4) route_dz_kernel<4><<<blocks, threads, 0, s>>>(a);
  else if (V <= 8) route_dz_kernel<8><<<blocks, threads, 0, s>>>(a);
  else route_dz_kernel<16><<<blocks, threads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_join_planes(const float* planes, int n, int64_t elems, void* dW, int grad_dtype, bool accumulate,
                               cudaStream_t s) {
  const int64_t vecs = elems / 4;
  return launch_after(join_planes_kernel, (unsigned)((vecs + 255) / 256), 256, 0, s,
                      reinterpret_cast<const float4*>(planes), n, vecs, dW, grad_dtype == MOE_F32, accumulate);
}

}  // namespace moe
