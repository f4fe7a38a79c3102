// Router backward: the gradient of the logits from the gradients of the
// gates, per token (half a warp; a warp for the dense softmax pass), and what
// joins the split weight gradient.
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
// Only selected experts have a gradient, except under an unnormalised softmax
// (normalised gates depend on ratios of the selected scores alone, so their
// softmax is taken relative to the largest selected logit). So a CTA zeroes a
// tile of 16 tokens in shared memory, half a warp per token works out its slots
// and scatters them, and the tile is written out both ways in 16-byte vectors.
// What bounds it is the chain launch - slot loads - scatter - stores:
// 4096 tokens of 256 experts take 5.6 us (4 MB of dz written; 11.5 us with a warp
// per token that held all experts in registers), 8192 of 63 under an unnormalised
// softmax, which reads all logits, 7 us.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

template <int W>
MOE_DEV float gsum(float v) {  // over W neighbouring lanes
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
template <int W>
MOE_DEV float gmax(float v) {
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

constexpr int kDzTokens = 16;  // tokens of a CTA: 32-byte runs of the transposed dz
constexpr int kDzSlots = 16;   // lanes of a token
constexpr int kDzThreads = kDzTokens * kDzSlots;
static_assert(kMaxTopK <= kDzSlots && kRouteTables <= kDzThreads, "a slot per lane, a table entry per thread");

// kDense: unnormalised softmax, where every expert's logit has a gradient.
template <bool kDense>
__global__ void __launch_bounds__(kDzThreads) route_dz_kernel(const __grid_constant__ RouteDzArgs a) {
  griddep_launch_dependents();
  extern __shared__ float4 dz_smem[];
  float* tile = reinterpret_cast<float*>(dz_smem);  // [token][expert], pitch ld
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && tid < kRouteTables) a.tables[tid] = a.table_values[tid];
  const int N = a.N, k = a.k, ld = (int)a.ld;
  const int64_t t0 = (int64_t)blockIdx.x * kDzTokens;
  const int w = tid / kDzSlots, slot = tid % kDzSlots;
  const int64_t t = t0 + w;
  const bool live = t < a.T && slot < k;
  int e = live ? __ldg(a.idx + t * k + slot) : -1;  // -1: none
  if (live && (e < 0 || e >= N)) {
    set_status(a.status, MOE_DEV_BAD_EXPERT);
    e = -1;
  }
  const float z = e >= 0 ? __ldg(a.logits + t * N + e) : -INFINITY;
  for (int i = tid; i < kDzTokens * ld / 4; i += kDzThreads) dz_smem[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  // (the other half of the warp is another token)
  const unsigned same = __match_any_sync(0xffffffffu, (w & 1) << 16 | (e & 0xffff));
  const bool first = e >= 0 && (tid & 31) == __ffs(same) - 1;  // the expert's first slot
  float dG = 0.f;
  if (a.slot_pos) {
    // the gradient of the slot's gate is that of the row the dispatch gave it:
    // slot_pos lists the token's rows by ascending expert
    int rank = 0;
    for (int i = 0; i < k; ++i) {
      const int ei = __shfl_sync(0xffffffffu, first ? e : -1, i, kDzSlots);
      rank += ei >= 0 && ei < e;
    }
    if (first) {
      const int32_t row = __ldg(a.slot_pos + t * k + rank);
      if (row >= 0 && row < a.T * k) dG = __ldg(a.dgates + row);
    }
  } else if (e >= 0) {
    dG = __ldg(a.dgates + t * k + slot);
  }
  float sc = 0.f, slope = 1.f;  // the score (up to Z) and what its logit's gradient takes from it
  if (a.score_fn == MOE_SIGMOID) {
    sc = e >= 0 ? 1.f / (1.f + expf(-z)) : 0.f;
    slope = sc * (1.f / (1.f + expf(z)));  // 1 - s without its cancellation
  } else if (!kDense) {
    const float m = gmax<kDzSlots>(z);
    sc = e >= 0 ? expf(z - m) : 0.f;
    slope = sc;
  }
  float ds = a.route_scale * dG;
  if (a.normalize) {
    const float Z = gsum<kDzSlots>(sc), dot = gsum<kDzSlots>(dG * sc);
    ds = a.route_scale / Z * (dG - dot / Z);
  }
  float sum = 0.f;  // over the slots that name this expert
  for (int i = 0; i < k; ++i) {
    const int ei = __shfl_sync(0xffffffffu, e, i, kDzSlots);
    const float v = __shfl_sync(0xffffffffu, ds, i, kDzSlots);
    if (ei == e) sum += v;
  }
  __syncthreads();
  if (first) tile[w * ld + e] = kDense ? sum : sum * slope;
  __syncthreads();
  if constexpr (kDense) {
    // a warp per token: s_j (ds_j - sum ds_i s_i) over all experts
    const int lane = tid & 31;
    for (int i = tid / 32; i < kDzTokens && t0 + i < a.T; i += kDzThreads / 32) {
      const float* logits = a.logits + (t0 + i) * N;
      float* row = tile + i * ld;
      float m = -INFINITY, Z = 0.f, dot = 0.f;
      for (int j = lane; j < N; j += 32) m = fmaxf(m, __ldg(logits + j));
      m = gmax<32>(m);
      for (int j = lane; j < N; j += 32) {
        const float x = expf(__ldg(logits + j) - m);
        Z += x;
        dot = fmaf(x, row[j], dot);
      }
      const float inv = 1.f / gsum<32>(Z), mean = gsum<32>(dot) * inv;
      for (int j = lane; j < N; j += 32) row[j] = expf(__ldg(logits + j) - m) * inv * (row[j] - mean);
    }
    __syncthreads();
  }
  const int tokens = (int)(a.T - t0 < kDzTokens ? a.T - t0 : kDzTokens);
  if (a.dz) {  // (columns N .. ld - 1 are zero)
    float4* out = reinterpret_cast<float4*>(a.dz + t0 * ld);
    for (int i = tid; i < tokens * ld / 4; i += kDzThreads) out[i] = dz_smem[i];
    return;
  }
  uint4* out = reinterpret_cast<uint4*>(a.dz16 + t0 * ld);
  for (int i = tid; i < tokens * ld / 8; i += kDzThreads) {
    const float4 u = dz_smem[2 * i], v = dz_smem[2 * i + 1];
    out[i] = make_uint4(pack_bf16x2(u.x, u.y), pack_bf16x2(u.z, u.w), pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
  if (!a.dz16_t) return;
  for (int i = tid; i < 2 * N; i += kDzThreads) {
    const int n = i >> 1, c = (i & 1) * 8;
    if (c >= tokens) continue;  // eight that start inside T may end in the row's padding
    const float* x = tile + c * ld + n;
    *reinterpret_cast<uint4*>(a.dz16_t + n * a.ld_t + t0 + c) =
        make_uint4(pack_bf16x2(x[0], x[ld]), pack_bf16x2(x[2 * ld], x[3 * ld]), pack_bf16x2(x[4 * ld], x[5 * ld]),
                   pack_bf16x2(x[6 * ld], x[7 * ld]));
  }
}

// dW = sum over the planes in order, rounded once (or added to an fp32 dW): two
// planes of 256 x 7168 4.7 us, mostly the launch and one round of loads from L2.
__global__ void __launch_bounds__(256) join_planes_kernel(const float4* planes, int n, int64_t vecs, void* dW, int f32,
                                                          int accumulate) {
  griddep_wait();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= vecs) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int q = 0; q < n; ++q) {
    const float4 w = planes[q * vecs + i];
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
  const size_t smem = (size_t)kDzTokens * a.ld * 4;
  if (a.score_fn == MOE_SOFTMAX && !a.normalize) route_dz_kernel<true><<<blocks, kDzThreads, smem, s>>>(a);
  else route_dz_kernel<false><<<blocks, kDzThreads, smem, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_join_planes(const float* planes, int n, int64_t elems, void* dW, int grad_dtype, bool accumulate,
                               cudaStream_t s) {
  const int64_t vecs = elems / 4;
  return launch_after(join_planes_kernel, (unsigned)((vecs + 255) / 256), 256, 0, s,
                      reinterpret_cast<const float4*>(planes), n, vecs, dW, grad_dtype == MOE_F32, accumulate);
}

}  // namespace moe
