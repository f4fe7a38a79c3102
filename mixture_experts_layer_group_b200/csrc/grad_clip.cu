// Global gradient norm over many tensors, and clipping.
//
// The tensors are cut into 64 KB chunks; a fixed grid of CTAs strides over
// them, so every CTA sums the same chunks in the same order and the result
// has the same bits each time. Squares are summed in fp32 over the 4 or 8
// values of one 16-byte vector and then in fp64; a vector whose sum leaves
// fp32's comfortable range is summed again in fp64. Both kernels are bound by
// HBM: one read for the norm, one read and one write for the scaling (none
// where a gradient in place needs no clipping). The scaling runs over the
// chunks backwards, so that what the norm read last comes from L2.
// The tensor table travels as a kernel parameter: nothing is copied, and a
// captured graph keeps its own.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunkBytes = 64 * 1024;
constexpr int kSmallTable = 64, kLargeTable = 512;  // tensors of one launch
constexpr int kMaxCtas = 148 * 8;
constexpr int kUnroll = 4;                          // 16-byte loads in flight per thread

template <int CAP>
struct Table {
  const uint8_t* src[CAP];
  uint8_t* dst[CAP];
  int64_t numel[CAP];
  int32_t chunk0[CAP + 1];  // chunks before tensor i
  uint8_t f32[CAP];
  int n;
};

struct Chunk {
  const uint8_t* src;
  uint8_t* dst;
  int64_t count;  // elements
  bool f32;
};

template <int CAP>
MOE_DEV Chunk chunk_of(const Table<CAP>& t, int c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.chunk0[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  const bool f32 = t.f32[lo];
  const int64_t per = kChunkBytes / (f32 ? 4 : 2), at = (int64_t)(c - t.chunk0[lo]) * per, left = t.numel[lo] - at;
  return Chunk{t.src[lo] + at * (f32 ? 4 : 2), t.dst[lo] + at * (f32 ? 4 : 2), left < per ? left : per, f32};
}

template <bool F32>
MOE_DEV float element(const uint8_t* p, int64_t i) {
  if (F32) return reinterpret_cast<const float*>(p)[i];
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}
template <bool F32>
MOE_DEV void put_element(uint8_t* p, int64_t i, float v) {
  if (F32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

template <bool F32>
MOE_DEV double square_sum(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[F32 ? 4 : 8], s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F32) {
      f[i] = __uint_as_float(w[i]);
    } else {
      const float2 p = unpack_bf16x2(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 8); ++i) s = fmaf(f[i], f[i], s);
  if (s > 1e-30f && s < 1e38f) return (double)s;
  double d = 0.0;  // tiny, huge or not finite
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 8); ++i) d = fma((double)f[i], (double)f[i], d);
  return d;
}

// The chunk's 16-byte vectors start at element `head` of the chunk.
MOE_DEV int64_t head_of(const uint8_t* p, int64_t count, int elem) {
  const int64_t h = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / elem;
  return h < count ? h : count;
}

template <bool F32>
MOE_DEV double chunk_square_sum(const Chunk& c) {
  constexpr int P = F32 ? 4 : 8;
  const int64_t head = head_of(c.src, c.count, 16 / P), vecs = (c.count - head) / P;
  const uint4* v = reinterpret_cast<const uint4*>(c.src + head * (16 / P));
  double sum = 0.0;
  int64_t i = threadIdx.x;
  for (; i + (kUnroll - 1) * kThreads < vecs; i += kUnroll * kThreads) {
    uint4 x[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) x[j] = __ldg(v + i + j * kThreads);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) sum += square_sum<F32>(x[j]);
  }
  for (; i < vecs; i += kThreads) sum += square_sum<F32>(__ldg(v + i));
  const int64_t tail = head + vecs * P;
  // at most 7 elements on each side
  if ((int64_t)threadIdx.x < head) {
    const double x = element<F32>(c.src, threadIdx.x);
    sum = fma(x, x, sum);
  }
  if (tail + (int64_t)threadIdx.x < c.count) {
    const double x = element<F32>(c.src, tail + threadIdx.x);
    sum = fma(x, x, sum);
  }
  return sum;
}

// Sum over the block, in a fixed order; valid in thread 0.
MOE_DEV double block_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
  return s;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) square_sum_kernel(const __grid_constant__ Table<CAP> t,
                                                              double* __restrict__ part) {
  griddep_launch_dependents();
  double sum = 0.0;
  for (int c = blockIdx.x; c < t.chunk0[t.n]; c += gridDim.x) {
    const Chunk ch = chunk_of(t, c);
    sum += ch.f32 ? chunk_square_sum<true>(ch) : chunk_square_sum<false>(ch);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) sum_parts_kernel(const double* __restrict__ part, int64_t n,
                                                             double* __restrict__ sumsq) {
  griddep_launch_dependents();
  griddep_wait();
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) sum += part[i];
  sum = block_sum(sum);
  if (threadIdx.x == 0) *sumsq = sum;
}

template <bool F32>
MOE_DEV uint4 scaled(uint4 v, float c) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F32) {
      w[i] = __float_as_uint(__uint_as_float(w[i]) * c);
    } else {
      const float2 p = unpack_bf16x2(w[i]);
      w[i] = pack_bf16x2(p.x * c, p.y * c);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F32>
MOE_DEV void scale_chunk(const Chunk& c, float coef) {
  constexpr int P = F32 ? 4 : 8;
  if ((reinterpret_cast<uintptr_t>(c.src) ^ reinterpret_cast<uintptr_t>(c.dst)) & 15u) {
    // source and destination sit differently within 16 bytes: element by element
    for (int64_t i = threadIdx.x; i < c.count; i += kThreads) put_element<F32>(c.dst, i, element<F32>(c.src, i) * coef);
    return;
  }
  const int64_t head = head_of(c.src, c.count, 16 / P), vecs = (c.count - head) / P;
  const uint4* v = reinterpret_cast<const uint4*>(c.src + head * (16 / P));
  uint4* o = reinterpret_cast<uint4*>(c.dst + head * (16 / P));
  int64_t i = threadIdx.x;
  for (; i + (kUnroll - 1) * kThreads < vecs; i += kUnroll * kThreads) {
    uint4 x[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) x[j] = v[i + j * kThreads];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) o[i + j * kThreads] = scaled<F32>(x[j], coef);
  }
  for (; i < vecs; i += kThreads) o[i] = scaled<F32>(v[i], coef);
  const int64_t tail = head + vecs * P;
  if ((int64_t)threadIdx.x < head) put_element<F32>(c.dst, threadIdx.x, element<F32>(c.src, threadIdx.x) * coef);
  if (tail + (int64_t)threadIdx.x < c.count)
    put_element<F32>(c.dst, tail + threadIdx.x, element<F32>(c.src, tail + threadIdx.x) * coef);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ Table<CAP> t,
                                                        const double* __restrict__ sumsq, float max_norm,
                                                        float* __restrict__ norm_out) {
  griddep_wait();
  const double norm = sqrt(*sumsq);
  // a norm that is not finite leaves the gradients as they are
  const bool clip = norm > (double)max_norm && isfinite(norm);
  const float coef = clip ? (float)((double)max_norm / norm) : 1.f;
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const int total = t.chunk0[t.n];
  for (int c = blockIdx.x; c < total; c += gridDim.x) {
    const Chunk ch = chunk_of(t, total - 1 - c);
    if (!clip && ch.src == ch.dst) continue;
    if (ch.f32) scale_chunk<true>(ch, coef);
    else scale_chunk<false>(ch, coef);
  }
}

// Runs `go(table, chunks, tensors before it)` over batches of the tensors.
template <int CAP, class Go>
moe_status for_batches(const moe_grad_tensor* x, int32_t n, Go go) {
  for (int32_t i = 0; i < n; i += CAP) {
    Table<CAP> t;
    t.n = 0;
    int64_t chunks = 0;
    for (int32_t j = i; j < n && j < i + CAP; ++j) {
      if (x[j].numel == 0) continue;
      const int64_t per = kChunkBytes / (x[j].dtype == MOE_F32 ? 4 : 2);
      t.src[t.n] = static_cast<const uint8_t*>(x[j].src);
      t.dst[t.n] = static_cast<uint8_t*>(x[j].dst ? x[j].dst : const_cast<void*>(x[j].src));
      t.numel[t.n] = x[j].numel;
      t.f32[t.n] = x[j].dtype == MOE_F32;
      t.chunk0[t.n++] = (int32_t)chunks;
      chunks += (x[j].numel + per - 1) / per;
      if (chunks > (1ll << 31) - 1) return MOE_ERR_UNSUPPORTED;
    }
    t.chunk0[t.n] = (int32_t)chunks;
    if (t.n == 0) continue;
    const cudaError_t e = go(t, (int)chunks);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return MOE_OK;
}

moe_status check_tensors(const moe_grad_tensor* x, int32_t n) {
  if (n < 0 || (n > 0 && !x)) return MOE_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i) {
    if (x[i].numel < 0 || (x[i].dtype != MOE_F32 && x[i].dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
    if (x[i].numel == 0) continue;
    const uintptr_t mask = x[i].dtype == MOE_F32 ? 3u : 1u;
    if (!x[i].src || (reinterpret_cast<uintptr_t>(x[i].src) & mask) || (reinterpret_cast<uintptr_t>(x[i].dst) & mask))
      return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

int ctas(int chunks) { return chunks < kMaxCtas ? chunks : kMaxCtas; }

template <int CAP>
moe_status norm_batches(const moe_grad_tensor* x, int32_t n, double* part, int64_t* parts, cudaStream_t s) {
  return for_batches<CAP>(x, n, [&](const Table<CAP>& t, int chunks) {
    square_sum_kernel<CAP><<<ctas(chunks), kThreads, 0, s>>>(t, part + *parts);
    *parts += ctas(chunks);
    return cudaGetLastError();
  });
}

template <int CAP>
moe_status clip_batches(const moe_grad_tensor* x, int32_t n, const double* sumsq, float max_norm, float* norm_out,
                        bool* launched, cudaStream_t s) {
  return for_batches<CAP>(x, n, [&](const Table<CAP>& t, int chunks) {
    const cudaError_t e =
        launch_after(clip_kernel<CAP>, ctas(chunks), kThreads, s, t, sumsq, max_norm, *launched ? nullptr : norm_out);
    *launched = true;
    return e;
  });
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_grad_norm_workspace_size(int32_t n, size_t* bytes) {
  if (n < 0 || !bytes) return MOE_ERR_INVALID_ARG;
  const size_t batches = n <= kSmallTable ? 1 : ((size_t)n + kLargeTable - 1) / kLargeTable;
  *bytes = align256(batches * kMaxCtas * sizeof(double));
  return MOE_OK;
}

moe_status moe_grad_norm(const moe_grad_tensor* tensors, int32_t n, double* sumsq, void* ws, size_t ws_bytes,
                         void* stream) {
  moe_status st = check_tensors(tensors, n);
  if (st != MOE_OK) return st;
  if (!sumsq || (reinterpret_cast<uintptr_t>(sumsq) & 7u)) return MOE_ERR_INVALID_ARG;
  size_t need = 0;
  moe_grad_norm_workspace_size(n, &need);
  if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u)) return MOE_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = wait_host_outputs(ws, s);
  if (e != cudaSuccess) return cuda_fail(e);
  double* part = static_cast<double*>(ws);
  int64_t parts = 0;
  st = n <= kSmallTable ? norm_batches<kSmallTable>(tensors, n, part, &parts, s)
                        : norm_batches<kLargeTable>(tensors, n, part, &parts, s);
  if (st != MOE_OK) return st;
  e = launch_after(sum_parts_kernel, 1, kThreads, s, part, parts, sumsq);
  if (e == cudaSuccess) e = note_device_use(ws, s);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status moe_grad_clip(const moe_grad_tensor* tensors, int32_t n, const double* sumsq, float max_norm,
                         float* norm_out, void* stream) {
  moe_status st = check_tensors(tensors, n);
  if (st != MOE_OK) return st;
  if (!sumsq || (reinterpret_cast<uintptr_t>(sumsq) & 7u) || (reinterpret_cast<uintptr_t>(norm_out) & 3u) ||
      !(max_norm >= 0.f))
    return MOE_ERR_INVALID_ARG;
  bool launched = false;
  cudaStream_t s = (cudaStream_t)stream;
  st = n <= kSmallTable ? clip_batches<kSmallTable>(tensors, n, sumsq, max_norm, norm_out, &launched, s)
                        : clip_batches<kLargeTable>(tensors, n, sumsq, max_norm, norm_out, &launched, s);
  if (st != MOE_OK) return st;
  if (!launched && norm_out) {  // no gradients: the norm alone
    Table<kSmallTable> t;
    t.n = 0;
    t.chunk0[0] = 0;
    const cudaError_t e = launch_after(clip_kernel<kSmallTable>, 1, kThreads, s, t, sumsq, max_norm, norm_out);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return MOE_OK;
}

}  // extern "C"
