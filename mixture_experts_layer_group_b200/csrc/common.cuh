// Device helpers shared by the sm_100a kernels: mbarriers with bounded
// waits, TMA tile loads, tcgen05 (tensor memory + UMMA) wrappers, bf16 and
// small warp utilities. Inline PTX only; no library kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "../../include/moe_b200.h"

#define MOE_DEV __device__ __forceinline__

namespace moe {

// Pipeline waits give up after this long (ns of %globaltimer) and report
// MOE_DEV_WAIT_TIMEOUT instead of hanging the GPU.
constexpr uint64_t kWaitLimitNs = 1000ull * 1000ull * 1000ull;

MOE_DEV uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16-byte shared-memory load / store through the shared state space.
MOE_DEV uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
MOE_DEV void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

MOE_DEV uint64_t global_timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

MOE_DEV uint32_t lane_id() { return threadIdx.x & 31u; }

// The warp's index within its block, in a form that the compiler keeps in
// uniform registers (as it then does with what follows from it).
MOE_DEV int uniform_warp_id() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

// True in exactly one lane of a converged warp. The operands of a tensor-core
// instruction are uniform registers: issued by a lane picked this way inside
// warp-uniform code, their values are computed there; inside a branch on the
// lane index every operand is first moved over from a thread's register,
// which made issuing a pair MMA about as long as its 128 cycles of work.
MOE_DEV bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// ---------------------------------------------------------------- mbarrier --

MOE_DEV void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}

MOE_DEV void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

MOE_DEV void mbar_arrive(uint64_t* bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(
                   smem_u32(bar))
               : "memory");
}

MOE_DEV void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(bytes)
      : "memory");
}

MOE_DEV bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Waits for the phase of `bar` with the given parity to complete. Returns
// false (and leaves the barrier untouched) once kWaitLimitNs has passed or
// *abort became nonzero; the caller then unwinds.
MOE_DEV bool mbar_wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) return false;
    }
  }
}

// ----------------------------------------------------------------- cluster --

MOE_DEV uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Address of the same shared-memory location in CTA `rank` of the cluster.
MOE_DEV uint32_t map_to_rank(uint32_t smem_addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
  return r;
}

// 4-byte store into shared memory of a CTA of the cluster that completes 4
// transaction bytes on an mbarrier of that CTA (its complete_tx has release
// semantics at cluster scope). The issuing thread does not wait for it.
MOE_DEV void st_async_u32(uint32_t cluster_addr, uint32_t v, uint32_t bar_cluster) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(cluster_addr),
               "r"(v), "r"(bar_cluster)
               : "memory");
}

MOE_DEV bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait_bounded for barriers that other CTAs of the cluster arrive on.
MOE_DEV bool mbar_wait_cluster_bounded(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) return false;
    }
  }
}

// Barrier across all threads of both CTAs of the cluster.
MOE_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// --------------------------------------------------------------------- TMA --

MOE_DEV void tma_prefetch_desc(const void* tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}

// 2-D tiled load of box {inner c0, outer c1} into shared memory, completing
// transaction bytes on `bar`. c0 is an element index along the innermost
// (contiguous) dimension and must be a multiple of 16 bytes' worth of
// elements; every caller passes multiples of 64 bf16 elements.
MOE_DEV void tma_load_2d(void* smem_dst, const void* tmap, uint64_t* bar, int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// 2-D tiled load with an L2 cache-policy hint (createpolicy result).
MOE_DEV void tma_load_2d_hint(void* smem_dst, const void* tmap, uint64_t* bar, int32_t c0,
                              int32_t c1, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}

// The same for a 3-D tensor map (c0 innermost).
MOE_DEV void tma_load_3d_hint(void* smem_dst, const void* tmap, uint64_t* bar, int32_t c0, int32_t c1, int32_t c2,
                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

// 2-D tiled load issued by either CTA of a CTA pair: data lands in this CTA's
// shared memory and the transaction bytes complete on `bar_cluster`, an
// mbarrier of the pair's first CTA (cluster address). No multicast.
MOE_DEV void tma_load_2d_pair(void* smem_dst, const void* tmap, uint32_t bar_cluster, int32_t c0,
                              int32_t c1, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar_cluster), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}

// The same for a 3-D tensor map (c0 innermost).
MOE_DEV void tma_load_3d_pair(void* smem_dst, const void* tmap, uint32_t bar_cluster, int32_t c0, int32_t c1,
                              int32_t c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

// `bytes` contiguous bytes of this GPU's memory into shared memory, completing
// transaction bytes on `bar`; both addresses and the size are multiples of 16.
MOE_DEV void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem_dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// 2-D tiled store of a shared-memory box to global memory (bulk group). The
// box start (c0, c1) must be non-negative and c0 a multiple of 16 bytes'
// worth of elements; rows/columns beyond the tensor are clipped.
MOE_DEV void tma_store_2d(const void* tmap, const void* smem_src, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(smem_u32(smem_src)), "r"(c0), "r"(c1)
               : "memory");
}
MOE_DEV void bulk_commit_group() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Waits until at most N committed bulk groups still read their shared-memory source.
template <int N>
MOE_DEV void bulk_wait_group_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
// Waits until every committed bulk group has completed.
MOE_DEV void bulk_wait_group_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Orders this thread's generic shared-memory writes before later async-proxy reads.
// Orders what this thread has seen of global memory before its later bulk copies from there.
MOE_DEV void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
MOE_DEV void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

MOE_DEV uint64_t policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

MOE_DEV uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

MOE_DEV uint64_t policy_evict_last() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// ----------------------------------------------------------------- tcgen05 --

// Allocates `ncols` tensor-memory columns (power of two >= 32) for this CTA;
// the base address is written to *dst_smem. Executed by one full warp.
MOE_DEV void tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
}

MOE_DEV void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

MOE_DEV void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// Pair versions (cta_group::2): executed by the same warp in both CTAs.
MOE_DEV void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
}

MOE_DEV void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

MOE_DEV void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// Programmatic dependent launch: a kernel launched with programmatic stream
// serialization may start before its predecessor ends; griddep_wait blocks
// until the predecessor grid has completed and its writes are visible (a
// no-op without the attribute); griddep_launch_dependents lets the
// dependent grid start once every CTA of this grid has called it or exited.
// (What a programmatic predecessor wrote is not read through __ldg or a const
// __restrict__ pointer: the compiler may take such data as constant for the whole
// kernel and move the read in front of the wait. Plain loads and this stay behind.)
MOE_DEV int32_t ld_after_wait(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
MOE_DEV void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
MOE_DEV void griddep_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// For a grid that does not wait for its predecessor although it reads what the
// grid before that wrote: the predecessor, which has waited for those writes,
// hands them on through a flag. One of its threads publishes after its
// griddep_wait and (where it lets them start early) before its dependents start, so
// the flag is set about when they look; the release and the acquire make what the
// wait made visible to the one visible to the other. The flag is zeroed by a kernel that
// had ended before the predecessor's wait did. Together about 1 us: a router backward
// of 46 us takes 47, one of 29 no more, a block backward of 59 us 60.
MOE_DEV void publish_waited(int* flag) { asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(flag) : "memory"); }
// False once kWaitLimitNs has passed without it.
MOE_DEV bool take_published(const int* flag) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    int32_t v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    if (v) return true;
    if (it == 0) t0 = global_timer_ns();
    else if ((it & 63u) == 0 && global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
}

MOE_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
MOE_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D[tmem] (+)= A[smem] * B[smem]^T, kind::f16 (bf16 inputs, fp32 accumulator),
// one 128 x N x 16 step. Issued by a single thread.
MOE_DEV void umma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Pair MMA (cta_group::2), issued by one thread of the pair's first CTA:
// D[256 x N] (+)= A[256 x 16] * B[N x 16]^T, A rows 0..127 and B rows
// 0..N/2-1 from this CTA's shared memory, the rest from the peer's at the
// same offsets; each CTA's TMEM holds its 128 rows of D.
MOE_DEV void umma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Pair MMA with A in tensor memory: D[256 x N] (+)= A[256 x 16] * B[N x 16]^T,
// A rows 0..127 in this CTA's TMEM lanes 0..127 at column a_tmem (16 bf16
// of a row packed two per 32-bit column, lower k in the low half) and rows
// 128..255 at the same address in the peer's; B as in umma_bf16_pair.
// N must be a multiple of 32.
MOE_DEV void umma_bf16_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives on the mbarrier at cluster address `bar_cluster` (this CTA's or the
// peer's) once the pair MMAs issued so far by this thread have completed.
MOE_DEV void umma_commit_pair(uint32_t bar_cluster) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar_cluster)
               : "memory");
}

// Arrives on the mbarrier at the same shared-memory offset in both CTAs of
// the pair once the pair MMAs issued so far by this thread have completed.
MOE_DEV void umma_commit_pair_both(uint32_t bar_smem) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(bar_smem), "h"((uint16_t)3) : "memory");
}

// Arrives on `bar` once every tcgen05 operation issued so far by this thread
// has completed.
MOE_DEV void umma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

// Shared-memory matrix descriptor for a K-major operand tile laid out by a
// 128-byte-swizzled TMA load: rows of 64 bf16 (128 B), 8-row swizzle atoms
// of 1024 B stacked contiguously. Fields (sm_100 layout): start address
// >> 4 in bits [0,14); leading byte offset >> 4 in [16,30) (unused for
// swizzled K-major, set to 1); stride byte offset >> 4 in [32,46) (1024 B
// between 8-row groups); version 1 in [46,48); swizzle mode 2 (128 B) in
// [61,64). Advancing K by 16 elements inside the 128-byte row adds 32 B to
// the start address.
MOE_DEV uint64_t smem_desc_sw128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1u << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// The same for an MN-major operand tile: 128-byte rows hold 64 consecutive
// elements of the M (or N) dimension at one k, 8 rows of consecutive k form a
// 1024-byte swizzle atom. Leading byte offset: from one 64-element chunk of
// M (N) to the next (`chunk_bytes`, the bytes of a 64 x K box); stride byte
// offset: from 8 k to the next 8 (1024 B). Advancing K by 16 elements adds
// 2048 B to the start address.
MOE_DEV uint64_t smem_desc_sw128_mn(uint32_t smem_addr, uint32_t chunk_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(chunk_bytes >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// Instruction descriptor, kind::f16: fp32 accumulator (bits [4,6) = 1), A and
// B bf16 (bits [7,10) and [10,13) = 1), both K-major (bits 15, 16 = 0),
// N >> 3 in bits [17,23), M >> 4 in bits [24,29).
__host__ __device__ constexpr uint32_t idesc_bf16_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// Instruction-descriptor bits for an MN-major A or B operand.
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;

// 32 lanes x 32 consecutive fp32 columns from tensor memory; thread i of the
// warp receives row (lane base + i). The caller issues tmem_wait_ld() before
// reading the registers.
MOE_DEV void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// 16 lanes x 256 bits, repeated over 4 column groups: thread i receives, for
// column group r (columns 8r .. 8r + 7 from taddr), r[4r + 0..1] = lane
// (base + i / 4), columns 8r + 2 (i % 4) + 0..1, and r[4r + 2..3] = lane
// (base + 8 + i / 4), the same columns (the m16n8 accumulator layout).
MOE_DEV void tmem_ld16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Four 8 x 8 bf16 matrices, stored transposed: thread i holds element pair
// (row i / 4, columns 2 (i % 4) + 0..1) of matrix m in register m; thread
// 8 m + k gives the shared-memory address of stored row k of matrix m, which
// receives column k (16 bytes).
MOE_DEV void stmatrix_x4_trans(uint32_t smem_addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_addr),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}

// The mirror of stmatrix_x4_trans: thread 8 m + k gives the address of stored
// row k of matrix m; thread i receives the pair (stored columns i / 4, stored
// rows 2 (i % 4) + 0..1) of matrix m in register m.
MOE_DEV void ldmatrix_x4_trans(uint32_t smem_addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(smem_addr)
               : "memory");
}

MOE_DEV void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 32 lanes x 32 consecutive 32-bit columns to tensor memory: thread i of the
// warp writes r[0..31] to row (lane base + i). The caller issues
// tmem_wait_st() before signalling that the columns are written.
MOE_DEV void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16,"
      " %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
MOE_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------------ values --

template <typename T>
MOE_DEV float to_f32(T v);
template <>
MOE_DEV float to_f32<float>(float v) { return v; }
template <>
MOE_DEV float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

MOE_DEV uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

MOE_DEV float silu_f32(float g) { return g / (1.0f + __expf(-g)); }

// Two fp32 values in one 64-bit register pair, and their packed arithmetic
// (each lane rounded as the scalar operation rounds it).
MOE_DEV uint64_t f32x2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
MOE_DEV void split_f32x2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
MOE_DEV uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
MOE_DEV uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
MOE_DEV uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
MOE_DEV uint64_t bf16x2_to_f32x2(uint32_t v) { return f32x2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
MOE_DEV uint32_t f32x2_to_bf16x2(uint64_t v) {
  float lo, hi;
  split_f32x2(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

// sigma(g) = 1 / (1 + 2^(-g log2 e)) of N pairs, by the hardware's exponential
// and reciprocal; 0 where the power overflows.
template <int N>
MOE_DEV void sigmoid_f32x2(const uint64_t (&g)[N], uint64_t (&s)[N]) {
  float x[N], y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) split_f32x2(mul_f32x2(g[i], f32x2(-1.4426950408889634f, -1.4426950408889634f)), x[i], y[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x[i]));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(y[i]));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) split_f32x2(add_f32x2(f32x2(x[i], y[i]), f32x2(1.0f, 1.0f)), x[i], y[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x[i]));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(y[i]));
    s[i] = f32x2(x[i], y[i]);
  }
}
MOE_DEV float2 unpack_bf16x2(uint32_t v) { return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v)); }

// silu(g) = g sigma(g) with sigma(g) = (1 + tanh(g / 2)) / 2 from the
// hardware tanh approximation (one special-function op). tanh.approx has a
// relative error near 2^-11, so sigma is off by at most about 2^-12 absolute
// and silu by |g| 2^-12: a fraction of the bf16 rounding of the result where
// g > 0, and small in norm where silu(g) is itself near zero.
MOE_DEV float silu_tanh(float g) {
  float t;
  asm("tanh.approx.f32 %0, %1;" : "=f"(t) : "f"(0.5f * g));
  const float hg = 0.5f * g;
  return fmaf(hg, t, hg);
}

MOE_DEV void set_status(unsigned* status, unsigned bits) {
  if (status) atomicOr(status, bits);
}

// Bounds checks of the debug build (-DMOE_DEBUG_BOUNDS): MOE_IN_BOUNDS(cond,
// status) is cond, and when cond is false it also records MOE_DEV_BOUNDS, so
// the caller skips the access it guards. The release build compiles it to
// true: its indices are correct by construction, and the debug build's test
// checks that no check fires on the same inputs.
#ifdef MOE_DEBUG_BOUNDS
#define MOE_IN_BOUNDS(cond, status) ((cond) ? true : (::moe::set_status((status), MOE_DEV_BOUNDS), false))
#else
#define MOE_IN_BOUNDS(cond, status) true
#endif

}  // namespace moe
