// common.cuh — device helpers shared by the SANTA++ kernels (sm_103a).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "santa.h"

namespace santa {

constexpr int kMaxGroup = 8;           // query heads per KV head supported by the kernels
constexpr int kChunk = 64;             // tokens per staged K/V chunk
constexpr int kMaxChunksPerSplit = 256;  // 64-token chunks one CTA may own
constexpr int kMaxTeamsPerCta = 1024;    // teams one CTA scores and samples
constexpr int kPubScores = 2048;         // scores a CTA can publish (its list region, 8 KiB)
constexpr int kMaxCluster = 16;          // CTAs per cluster (non-portable above 8)
constexpr int kMaxClustersPerUnit = 16;  // clusters serving one unit
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s: no copy of ours takes that long

__device__ __forceinline__ void set_status(int32_t* status, uint32_t bits) {
  if (status) atomicOr(reinterpret_cast<unsigned int*>(status), bits);
}

// bf16 pairs packed in a 32-bit word -> fp32 (bf16 is the top half of an fp32).
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf16_to_f32(uint16_t h) {
  return __uint_as_float(static_cast<uint32_t>(h) << 16);
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// ---------------------------------------------------------------- mbarrier + bulk copies

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count)
               : "memory");
}

// Programmatic dependent launch: the grid may be scheduled before the previous kernel in
// its stream has finished; grid_dependency_wait() blocks until that kernel has completed and
// its memory is visible (a no-op when the launch had no such dependency), and
// grid_launch_dependents() lets the next kernel of the stream be scheduled early.
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Split cluster barrier; every thread of every CTA of the cluster executes each once, in
// this order, with no other cluster barrier in between.  The arrive is relaxed: it orders no
// memory operations, so it may only announce that remote reads whose values the thread has
// already consumed are over (a returned load cannot observe a later store).
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// Barrier over `nthreads` threads (a multiple of 32) on named barrier `id` (1..15), which
// returns whether `pred` held for any of them.
__device__ __forceinline__ bool bar_red_or(int id, int nthreads, bool pred) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(pred)), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}
// Orders this thread's generic-proxy shared-memory writes before later async-proxy (bulk
// copy) accesses of the same bytes; a barrier must follow before the copy is issued.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Makes mbarrier initialisation visible to the asynchronous (bulk copy) proxy.
__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
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

// Waits for phase `parity` of `bar` to complete, for at most kWaitLimitNs.  Returns false
// (and the caller records SANTA_DEV_TIMEOUT) if the phase never completed.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t start = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - start > kWaitLimitNs) return false;
  }
  return true;
}

// One contiguous global -> shared bulk copy (TMA, non-tensor form) that completes `bytes`
// transaction bytes on `bar`.  dst, src and bytes must be multiples of 16.
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Address of the same shared-memory location in CTA `rank` of this cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t smem_addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
  return r;
}

// Stores to another CTA of the cluster that complete their bytes on that CTA's mbarrier:
// dst and bar are cluster addresses (cluster_addr); dst 16- (v4) or 8-byte (v2) aligned.
__device__ __forceinline__ void st_async_v4(uint32_t dst, float4 v, uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
      ::"r"(dst), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void st_async_v2(uint32_t dst, float a, float b, uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];"
      ::"r"(dst), "f"(a), "f"(b), "r"(bar)
      : "memory");
}

// Atomic add at GPU scope with acquire-release semantics: the caller's earlier writes (and
// those of its CTA, after a CTA barrier) are visible to whoever reads the sum later, and the
// writes of the earlier adders are visible to the caller afterwards.
__device__ __forceinline__ unsigned int atomic_add_acq_rel_gpu(unsigned int* addr, unsigned int v) {
  unsigned int old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
               : "=r"(old) : "l"(addr), "r"(v) : "memory");
  return old;
}

// Two-dimensional tensor copy global -> shared through a tensor map (TMA): the box at
// (x, y) (x the innermost coordinate, in elements) lands at dst and completes on bar.
__device__ __forceinline__ void tma_load_2d(void* dst, const void* tmap, int x, int y,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y),
        "r"(smem_u32(bar))
      : "memory");
}

// Bring a tensor-map descriptor (kernel parameter) into the descriptor cache ahead of its
// first use by a tensor copy.
__device__ __forceinline__ void prefetch_tensormap(const void* tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}

// ---------------------------------------------------------------- warp matrix fragments

// Four 8x8 b16 matrices from shared memory (row addresses given per lane).
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// Transpose of an 8x8 b16 matrix held one row-pair per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// D = A (16x16 bf16, row) * B (16x8 bf16, col) + C, fp32 accumulate.
__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two fp32 values as packed bf16 (round to nearest even): lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf16_lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 16-byte asynchronous global -> shared copy (L2 only), completed by cp_async_wait_all.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------- host: launch attributes

// Raises a kernel's dynamic shared-memory limit once per device (so that launches, including
// launches during CUDA-graph capture, make no attribute call).
template <typename Kernel>
inline cudaError_t ensure_dynamic_smem(Kernel* kernel, size_t bytes,
                                       std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// 2^x by the SFU's approximate instruction (relative error near 2^-22; results below 2^-126
// flush to zero, 2^-inf is 0)
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- warp reductions

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ---------------------------------------------------------------- ragged chunks

// The sequence that owns work slot `slot` of a ragged batch: the last b < batch with
// s(b) <= slot, s(b) = floor(cu[b] / per) + extra * b (0 if there is none).  cu[b] is clamped to
// [0, num_tokens], and any cu at all gives some b in [0, batch).  The whole warp calls it with
// the same arguments; 32 candidates per round.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int64_t num_tokens,
                                             int per, int extra, int64_t slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    bool below = lane == 0;
    if (lane > 0 && at < hi) {
      int64_t c = cu[at];
      c = c < 0 ? 0 : c > num_tokens ? num_tokens : c;
      below = c / per + static_cast<int64_t>(extra) * at <= slot;
    }
    const unsigned m = __ballot_sync(0xffffffffu, below);
    lo += (31 - __clz(m)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Sets SANTA_DEV_BAD_SEQLEN if cu is not non-decreasing within [0, num_tokens] (a search over
// such a cu may miss the sequence it concerns); by all threads of one block.
__device__ __forceinline__ void check_bounds(const int32_t* cu, int batch, int64_t num_tokens,
                                             int32_t* status) {
  for (int b = threadIdx.x; b < batch; b += blockDim.x)
    if (cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > num_tokens)
      set_status(status, SANTA_DEV_BAD_SEQLEN);
}

// ---------------------------------------------------------------- Philox4x32-10

// Counter-based generator of Salmon, Moraes, Dror and Shaw, "Parallel Random Numbers: As
// Easy as 1, 2, 3" (SC'11): ten rounds; each multiplies counter words 0 and 2 by the two
// round multipliers and mixes the high halves with words 1, 3 and the round key, which is
// advanced by the two Weyl increments before every round but the first.
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint2 k) {
#pragma unroll
  for (int round = 0; round < 10; ++round) {
    if (round > 0) {
      k.x += 0x9E3779B9u;
      k.y += 0xBB67AE85u;
    }
    const uint32_t hi0 = __umulhi(0xD2511F53u, c.x), lo0 = 0xD2511F53u * c.x;
    const uint32_t hi1 = __umulhi(0xCD9E8D57u, c.z), lo1 = 0xCD9E8D57u * c.z;
    c = make_uint4(hi1 ^ c.y ^ k.x, lo1, hi0 ^ c.w ^ k.y, lo0);
  }
  return c;
}

// The same generator with its rounds in a loop: a tenth of the instructions, for code that
// runs once per launch, where fetching the unrolled form costs more than the loop.
__device__ __forceinline__ uint4 philox4x32_10_compact(uint4 c, uint2 k) {
#pragma unroll 1
  for (int round = 0; round < 10; ++round) {
    const uint32_t hi0 = __umulhi(0xD2511F53u, c.x), lo0 = 0xD2511F53u * c.x;
    const uint32_t hi1 = __umulhi(0xCD9E8D57u, c.z), lo1 = 0xCD9E8D57u * c.z;
    c = make_uint4(hi1 ^ c.y ^ k.x, lo1, hi0 ^ c.w ^ k.y, lo0);
    k.x += 0x9E3779B9u;
    k.y += 0xBB67AE85u;
  }
  return c;
}

}  // namespace santa
