// Global gradient norm over many tensors, and clipping.
//
// The tensors are cut into 64 KB chunks; a fixed grid of CTAs strides over
// them, so every CTA sums the same chunks in the same order and the result
// has the same bits each time. Squares are summed in fp32 over the 16 or 32
// values a thread takes of one piece and then in fp64; values whose sum leaves
// fp32's comfortable range are summed again in fp64. Both kernels are bound by
// HBM: one read for the norm, one read and one write for the scaling (none
// where a gradient in place needs no clipping). Loads are bulk copies into a
// ring of 16 KB pieces, 96 KB per CTA and two CTAs per SM, because about 190
// KB in flight per SM are what it takes to read at the memory's rate: the norm of
// 2.8 GB takes 446 us (6.3 TB/s), where registers as the destination (four
// 16-byte loads per thread in flight) took 500; the scaling of the same, out of
// place, 900 us (6.3 TB/s of reads and writes). The scaling runs over the chunks backwards, so
// that what the norm read last comes from L2.
// The tensor table travels as a kernel parameter: nothing is copied, and a
// captured graph keeps its own.
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;                       // that compute; one more warp issues the loads
constexpr int kChunkBytes = 64 * 1024;
constexpr int kSmallTable = 64, kLargeTable = 512;  // tensors of one launch
constexpr int kMaxCtas = 148 * 2;
constexpr int kPiece = 16 * 1024;
constexpr int kSlots = 6;
constexpr int kRingBytes = kSlots * kPiece;

template <int CAP>
struct Table {
  const uint8_t* src[CAP];
  uint8_t* dst[CAP];
  int64_t numel[CAP];
  int32_t chunk0[CAP + 1];  // chunks before tensor i
  uint8_t f32[CAP];
  int n;
  int inplace;              // every dst is its src
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

// Sum of the squares of up to kVecs vectors, `stride` apart (the first
// `count`): in fp32 over the (at most 32) values, or, when that leaves fp32's
// comfortable range, in fp64.
constexpr int kVecs = kPiece / 16 / kThreads;
template <bool F32>
MOE_DEV void values_of(uint4 v, float (&f)[F32 ? 4 : 8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F32) {
      f[i] = __uint_as_float(w[i]);
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <bool F32>
MOE_DEV double square_sum(const uint4 (&v)[kVecs]) {
  float part[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float f[F32 ? 4 : 8];
    values_of<F32>(v[j], f);
    part[j] = f[0] * f[0];
#pragma unroll
    for (int i = 1; i < (F32 ? 4 : 8); ++i) part[j] = fmaf(f[i], f[i], part[j]);
  }
  static_assert(kVecs == 4, "summed in pairs");
  const float s = (part[0] + part[1]) + (part[2] + part[3]);
  if (s > 1e-30f && s < 1e38f) return (double)s;
  double d = 0.0;  // tiny, huge or not finite
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float f[F32 ? 4 : 8];
    values_of<F32>(v[j], f);
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 8); ++i) d = fma((double)f[i], (double)f[i], d);
  }
  return d;
}

// Elements of the chunk before its first 16-byte boundary.
MOE_DEV int64_t head_of(const Chunk& c) {
  const int elem = c.f32 ? 4 : 2;
  const int64_t h = (int64_t)((16 - (reinterpret_cast<uintptr_t>(c.src) & 15u)) & 15u) / elem;
  return h < c.count ? h : c.count;
}
// Its 16-byte vectors after them, 4 or 8 elements each.
MOE_DEV int vecs_of(const Chunk& c, int64_t head) { return (int)((c.count - head) / (c.f32 ? 4 : 8)); }

// What the load warp tells the others about a slot of the ring.
enum Kind : int { kVecF32 = 0, kVecBf16 = 1, kElemF32 = 2, kElemBf16 = 3, kEnd = 4 };
struct Piece {
  const uint8_t* src;  // element kinds: read from memory, nothing was loaded
  uint8_t* dst;
  int64_t count;       // vectors or elements
  int kind;
};
struct Ring {
  uint64_t full[kSlots], empty[kSlots];
  Piece piece[kSlots];
  int abort_flag;
};

// The load warp walks the CTA's chunks and fills the ring with their vectors;
// edge(chunk, from, to) handles the up to 7 elements on each side, by its
// lanes, skip(chunk) leaves a chunk out and apart(chunk) hands it over whole, to
// be read element by element. The other warps call use(piece, data) for every
// piece as it lands: they neither search the table nor divide. False when a
// wait ran out (in the threads that saw it).
template <int CAP, class Skip, class Apart, class Use, class Edge>
MOE_DEV bool stream_chunks(const Table<CAP>& t, bool backwards, Skip skip, Apart apart, Use use, Edge edge) {
  extern __shared__ __align__(128) uint8_t ring_bytes[];
  __shared__ Ring ring;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&ring.full[s], 1);
      mbar_init(&ring.empty[s], kThreads / 32);
    }
    ring.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  uint32_t j = 0;  // pieces so far
  bool ok = true;
  if (warp == kThreads / 32) {
    const int total = t.chunk0[t.n];
    auto put = [&](const Piece& p, const uint8_t* load, uint32_t bytes) {  // lane 0
      const uint32_t s = j % kSlots;
      if (!mbar_wait_bounded(&ring.empty[s], ((j / kSlots) & 1u) ^ 1u, &ring.abort_flag)) return false;
      ++j;
      ring.piece[s] = p;
      if (bytes) {
        mbar_arrive_expect_tx(&ring.full[s], bytes);
        bulk_load(ring_bytes + s * kPiece, load, bytes, &ring.full[s]);
      } else {
        mbar_arrive(&ring.full[s]);
      }
      return true;
    };
    for (int c = blockIdx.x; c < total; c += gridDim.x) {
      const Chunk ch = chunk_of(t, backwards ? total - 1 - c : c);
      if (skip(ch)) continue;
      const int elem = ch.f32 ? 4 : 2;
      if (apart(ch)) {
        if (lane == 0) ok = put(Piece{ch.src, ch.dst, ch.count, ch.f32 ? kElemF32 : kElemBf16}, nullptr, 0);
      } else {
        const int64_t head = head_of(ch);
        const int bytes = vecs_of(ch, head) * 16;
        edge(ch, 0, head);
        edge(ch, head + bytes / elem, ch.count);
        if (lane == 0)
          for (int at = 0; ok && at < bytes; at += kPiece) {
            const int n = bytes - at < kPiece ? bytes - at : kPiece;
            const int64_t off = head * elem + at;
            ok = put(Piece{nullptr, ch.dst + off, n / 16, ch.f32 ? kVecF32 : kVecBf16}, ch.src + off, n);
          }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0);
      if (!ok) break;
    }
    if (lane == 0) {
      if (ok) ok = put(Piece{nullptr, nullptr, 0, kEnd}, nullptr, 0);
      if (!ok) {
        *reinterpret_cast<volatile int*>(&ring.abort_flag) = 1;
        int no_abort = 0;  // no load may be in flight when the block ends (else every piece has been waited for)
        for (uint32_t i = j > kSlots ? j - kSlots : 0; i < j; ++i)
          (void)mbar_wait_bounded(&ring.full[i % kSlots], (i / kSlots) & 1u, &no_abort);
      }
    }
    __syncwarp();
    return ok;
  }
  for (;; ++j) {
    const uint32_t s = j % kSlots;
    ok = mbar_wait_bounded(&ring.full[s], (j / kSlots) & 1u, &ring.abort_flag);
    if (!ok) {
      *reinterpret_cast<volatile int*>(&ring.abort_flag) = 1;
      break;
    }
    const Piece p = ring.piece[s];
    if (p.kind == kEnd) break;
    use(p, ring_bytes + s * kPiece);
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring.empty[s]);
  }
  return ok;
}

// Sum over the block, in a fixed order; valid in thread 0.
MOE_DEV double block_sum(double v) {
  __shared__ double part[kThreads / 32 + 1];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < blockDim.x / 32; ++i) s += part[i];
  return s;
}

template <bool F32>
MOE_DEV double piece_square_sum(const uint8_t* data, int64_t count) {
  uint4 v[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int at = threadIdx.x + i * kThreads;
    v[i] = at < count ? ld_shared_v4(smem_u32(data + at * 16)) : make_uint4(0, 0, 0, 0);
  }
  return square_sum<F32>(v);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads + 32) square_sum_kernel(const __grid_constant__ Table<CAP> t,
                                                                   double* __restrict__ part) {
  griddep_launch_dependents();
  double sum = 0.0;
  const bool ok = stream_chunks(
      t, false, [](const Chunk&) { return false; }, [](const Chunk&) { return false; },
      [&](const Piece& p, const uint8_t* data) {
        sum += p.kind == kVecF32 ? piece_square_sum<true>(data, p.count) : piece_square_sum<false>(data, p.count);
      },
      [&](const Chunk& c, int64_t from, int64_t to) {
        const int64_t i = from + (threadIdx.x & 31);
        if (i < to) {
          const double x = c.f32 ? element<true>(c.src, i) : element<false>(c.src, i);
          sum = fma(x, x, sum);
        }
      });
  if (!ok) sum = __longlong_as_double(0x7ff8000000000000ll);  // a load that never came: no norm
  sum = block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) sum_parts_kernel(const double* part, int64_t n, double* sumsq) {
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
MOE_DEV void scale_piece(const uint8_t* piece, int count, uint4* out, float coef) {
#pragma unroll
  for (int i = 0; i < kPiece / 16 / kThreads; ++i) {
    const int v = threadIdx.x + i * kThreads;
    if (v < count) out[v] = scaled<F32>(ld_shared_v4(smem_u32(piece + v * 16)), coef);
  }
}
template <bool F32>
MOE_DEV void scale_elements(const uint8_t* src, uint8_t* dst, int64_t from, int64_t to, int64_t step, float coef) {
  for (int64_t i = from; i < to; i += step) put_element<F32>(dst, i, element<F32>(src, i) * coef);
}

// A wait that runs out leaves chunks unscaled; norm_out then holds the mark
// MOE_NORM_INCOMPLETE instead of the norm. CTAs that give up write it with
// exchanges, and the one exchange that writes the norm puts the mark back when it
// was there already: whichever order they run in, the mark stays. (So it also stays
// from one call to the next, until the caller overwrites it.) `first`: this launch
// writes the norm; it is one of several when the tensors take more tables.
template <int CAP>
__global__ void __launch_bounds__(kThreads + 32) clip_kernel(const __grid_constant__ Table<CAP> t,
                                                             const double* sumsq, float max_norm, float* norm_out,
                                                             int first) {
  griddep_wait();
  const double norm = sqrt(*sumsq);
  // a norm that is not finite leaves the gradients as they are
  const bool clip = norm > (double)max_norm && isfinite(norm);
  const float coef = clip ? (float)((double)max_norm / norm) : 1.f;
  unsigned* out = reinterpret_cast<unsigned*>(norm_out);
  unsigned held = 0;
  if (out && first && blockIdx.x == 0 && threadIdx.x == 0) held = atomicExch(out, __float_as_uint((float)norm));
  bool ok = true;
  if (clip || !t.inplace)
    ok = stream_chunks(
        t, true, [&](const Chunk& c) { return !clip && c.src == c.dst; },
        [&](const Chunk& c) {  // source and destination sit differently within 16 bytes
          return ((reinterpret_cast<uintptr_t>(c.src) ^ reinterpret_cast<uintptr_t>(c.dst)) & 15u) != 0;
        },
        [&](const Piece& p, const uint8_t* data) {
          switch (p.kind) {
            case kVecF32: scale_piece<true>(data, (int)p.count, reinterpret_cast<uint4*>(p.dst), coef); break;
            case kVecBf16: scale_piece<false>(data, (int)p.count, reinterpret_cast<uint4*>(p.dst), coef); break;
            case kElemF32: scale_elements<true>(p.src, p.dst, threadIdx.x, p.count, kThreads, coef); break;
            default: scale_elements<false>(p.src, p.dst, threadIdx.x, p.count, kThreads, coef);
          }
        },
        [&](const Chunk& c, int64_t from, int64_t to) {
          const int64_t i = from + (threadIdx.x & 31);
          if (c.f32) scale_elements<true>(c.src, c.dst, i, to, 32, coef);
          else scale_elements<false>(c.src, c.dst, i, to, 32, coef);
        });
  if (out && (!ok || held == MOE_NORM_INCOMPLETE)) atomicExch(out, MOE_NORM_INCOMPLETE);
}

// Runs `go(table, chunks, tensors before it)` over batches of the tensors.
template <int CAP, class Go>
moe_status for_batches(const moe_grad_tensor* x, int32_t n, Go go) {
  for (int32_t i = 0; i < n; i += CAP) {
    Table<CAP> t;
    t.n = 0;
    t.inplace = 1;
    int64_t chunks = 0;
    for (int32_t j = i; j < n && j < i + CAP; ++j) {
      if (x[j].numel == 0) continue;
      const int64_t per = kChunkBytes / (x[j].dtype == MOE_F32 ? 4 : 2);
      t.src[t.n] = static_cast<const uint8_t*>(x[j].src);
      t.dst[t.n] = static_cast<uint8_t*>(x[j].dst ? x[j].dst : const_cast<void*>(x[j].src));
      t.inplace &= t.dst[t.n] == t.src[t.n];
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

// The shared-memory opt-in of a kernel, once per device.
template <auto kKernel>
cudaError_t allow_ring() {
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  done[dev] = e == cudaSuccess;
  return e;
}

int ctas(int chunks) { return chunks < kMaxCtas ? chunks : kMaxCtas; }

template <int CAP>
moe_status norm_batches(const moe_grad_tensor* x, int32_t n, double* part, int64_t* parts, cudaStream_t s) {
  return for_batches<CAP>(x, n, [&](const Table<CAP>& t, int chunks) {
    const cudaError_t e = allow_ring<square_sum_kernel<CAP>>();
    if (e != cudaSuccess) return e;
    square_sum_kernel<CAP><<<ctas(chunks), kThreads + 32, kRingBytes, s>>>(t, part + *parts);
    *parts += ctas(chunks);
    return cudaGetLastError();
  });
}

template <int CAP>
moe_status clip_batches(const moe_grad_tensor* x, int32_t n, const double* sumsq, float max_norm, float* norm_out,
                        bool* launched, cudaStream_t s) {
  return for_batches<CAP>(x, n, [&](const Table<CAP>& t, int chunks) {
    cudaError_t e = allow_ring<clip_kernel<CAP>>();
    if (e == cudaSuccess)
      e = launch_after(clip_kernel<CAP>, ctas(chunks), kThreads + 32, kRingBytes, s, t, sumsq, max_norm, norm_out,
                       (int)!*launched);
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
  e = launch_after(sum_parts_kernel, 1, kThreads, 0, s, part, parts, sumsq);
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
    t.inplace = 1;
    t.chunk0[0] = 0;
    cudaError_t e = allow_ring<clip_kernel<kSmallTable>>();
    if (e == cudaSuccess)
      e = launch_after(clip_kernel<kSmallTable>, 1, kThreads + 32, kRingBytes, s, t, sumsq, max_norm, norm_out, 1);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return MOE_OK;
}

}  // extern "C"
