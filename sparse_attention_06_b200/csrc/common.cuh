// common.cuh -- device helpers shared by the DSA kernels (sm_100a).
//
// Contents: the device error word, dtype loads for the generic CUDA-core path, bounded mbarrier
// waits, and thin inline-PTX wrappers for the Blackwell data-movement and tensor-core
// instructions used by the tcgen05 kernels (TMA tensor loads, cp.async, tcgen05.alloc / mma /
// commit / ld, fences).  Nothing here computes any part of the method.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dsa.h"

namespace dsa {

// ---------------------------------------------------------------------------------------------
// error word
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void raise_error(int* err, int bit) {
  if (err) atomicOr(err, bit);
}

// ---------------------------------------------------------------------------------------------
// element loads (generic path)
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ float bf16_bits_to_float(uint16_t b) {
  return __uint_as_float(((uint32_t)b) << 16);
}

__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
  __nv_fp8_e4m3 v;
  v.__x = b;
  return float(v);
}

__device__ __forceinline__ float load_elem(const void* base, int dtype, int64_t i) {
  if (dtype == DSA_F32) return static_cast<const float*>(base)[i];
  if (dtype == DSA_BF16) return bf16_bits_to_float(static_cast<const uint16_t*>(base)[i]);
  return e4m3_to_float(static_cast<const uint8_t*>(base)[i]);
}

// A quantised latent row's group scale: a power of two 2^e, -100 <= e <= 119.
__device__ __forceinline__ bool latent_scale_ok(float s) {
  const uint32_t b = __float_as_uint(s);
  return (b & 0x807FFFFFu) == 0u && (b >> 23) >= 27u && (b >> 23) <= 246u;
}

// Value of element i of pool row `row`, any cache dtype.
__device__ __forceinline__ float load_cached(const dsa_paged_cache& c, int64_t row, int i) {
  if (c.dtype == DSA_LATENT_E4M3) {
    const uint8_t* p = static_cast<const uint8_t*>(c.data) + row * 640;
    return i < 512 ? e4m3_to_float(p[i]) * c.scale[row * 4 + (i >> 7)]
                   : bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p + 512)[i - 512]);
  }
  const float v = load_elem(c.data, c.dtype, row * c.dim + i);
  return c.dtype == DSA_E4M3 ? v * c.scale[row] : v;
}

// Request and position of row t of a call's chunks; false for a row behind the last request, and
// for one whose request has bounds outside the call's (flagged).
__device__ __forceinline__ bool chunk_token(const dsa_chunks& c, int t, int* req, int* pos, int* err) {
  if (t >= c.num_tokens || t < c.cu_tokens[0] || t >= c.cu_tokens[c.num_reqs]) return false;
  int lo = 0, hi = c.num_reqs;  // cu_tokens[lo] <= t < cu_tokens[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c.cu_tokens[mid] <= t) lo = mid; else hi = mid;
  }
  const int first = c.cu_tokens[lo], end = c.cu_tokens[lo + 1], len = c.seq_len[lo];
  if (first < 0 || end > c.num_tokens || len > c.max_context || len < end - first) {
    raise_error(err, DSA_DEVERR_REQUEST);
    return false;
  }
  *req = lo;
  *pos = len - (end - t);
  return true;
}

// ---------------------------------------------------------------------------------------------
// order keys of scores (selection) and their digit histogram
// ---------------------------------------------------------------------------------------------
// Order-preserving 32-bit key of a score: a larger score has a larger key, -0.0 has the key of
// +0.0, and NaN gets the lowest key (0) with `is_nan` set.
__device__ __forceinline__ uint32_t order_key(float f, bool& is_nan) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) {
    is_nan = true;
    return 0u;
  }
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Histogram of order keys by their top kKeyDigitBits bits (sign, exponent and three mantissa
// bits: eight bins per binade), one row of kKeyBins counters per query.  The indexer adds its
// scores to it; the selection reads a row to place its threshold and clears it again.
constexpr int kKeyDigitBits = 12;
constexpr int kKeyBins = 1 << kKeyDigitBits;
__device__ __forceinline__ uint32_t key_digit(uint32_t key) { return key >> (32 - kKeyDigitBits); }

// ---------------------------------------------------------------------------------------------
// shared-memory addresses, mbarriers
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
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

// Default limit of a bounded wait, in SM cycles (about two seconds at 1.9 GHz); a wait that has
// not seen its phase complete by then gives up.
constexpr long long kWaitCycles = 4000000000LL;

// Bounded wait on an mbarrier phase.  Returns false (and raises DSA_DEVERR_TIMEOUT) when the
// phase did not complete within `limit` SM cycles, or when another role of this CTA already gave
// up (*abort_flag).
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, int* err,
                                          volatile int* abort_flag, long long limit = kWaitCycles) {
  if (mbar_try_wait(bar, parity)) return true;
  long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (abort_flag && *abort_flag) return false;
    if (clock64() - t0 > limit) {
      raise_error(err, DSA_DEVERR_TIMEOUT);
      if (abort_flag) *abort_flag = 1;
      return false;
    }
  }
}

// Warp-collective form: every lane waits, and the warp proceeds only if every lane saw the phase
// complete, so that a timeout never leaves a warp diverged before a .sync.aligned instruction.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err, volatile int* abort_flag) {
  const bool ok = mbar_wait(bar, parity, err, abort_flag);
  return __all_sync(0xFFFFFFFFu, ok);
}

// ---------------------------------------------------------------------------------------------
// programmatic dependent launch
// ---------------------------------------------------------------------------------------------
// A kernel launched with programmatic stream serialization may start while the previous kernel
// of the stream is still running; it must not touch global memory that kernel may write before
// griddep_wait() returns (which waits for that kernel's completion and memory flush).
// griddep_launch_dependents() lets the next kernel of the stream begin launching; it takes effect
// once every CTA of this grid has called it or exited.  Both are no-ops without the attribute.
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------------------------------------
// async-proxy fences, TMA, cp.async
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 2-D tiled TMA load (no multicast) into shared memory, completion counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_2d(void* smem_dst, const void* tmap, uint64_t* bar,
                                            int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// L2 cache policy that makes the lines a load brings in the first to be evicted: for data read once
// (keys streamed past a single query), so that they do not push out what the next kernel reads.
__device__ __forceinline__ uint64_t l2_policy_evict_first() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// tma_load_2d with an L2 cache-policy hint (a policy from createpolicy).
__device__ __forceinline__ void tma_load_2d_hint(void* smem_dst, const void* tmap, uint64_t* bar,
                                                 int32_t c0, int32_t c1, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}

// TMA gather of four rows (tile::gather4; 2-D tensor map whose box is one row high): columns
// [c0, c0 + box) of rows r0..r3 land as four consecutive box rows at smem_dst, completion counted
// on `bar` in bytes.  Rows outside the tensor read as zeros.  No multicast.
__device__ __forceinline__ void tma_gather4(void* smem_dst, const void* tmap, uint64_t* bar, int32_t c0,
                                            int32_t r0, int32_t r1, int32_t r2, int32_t r3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
      : "memory");
}

// Bring `bytes` (a multiple of 16) of global memory at a 16-byte aligned address into L2.
__device__ __forceinline__ void prefetch_l2_bulk(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<uint64_t>(src)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void prefetch_tmap(const void* tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}

// 4-byte cp.async (through L1), for scattered scalars.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Wait for every cp.async this thread issued, committed to a group or not.
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---------------------------------------------------------------------------------------------
// tcgen05 (5th-generation tensor cores, accumulators in tensor memory)
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* smem_slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(smem_slot)),
               "r"(ncols)
               : "memory");
}

__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A * B^T, kind::f16 (bf16/f16 inputs, f32 accumulate): umma_ss with A and B from
// shared-memory descriptors, umma_ts with A (M rows x 16 K) read from tensor memory, one row per
// lane, two consecutive K elements per 32-bit column.  Issue-lean forms for unrolled chains: the
// accumulate flag is a compile-time constant and there is no memory clobber (ordering against
// shared-memory writes comes from the fences and mbarrier waits around the chain, which are
// volatile asm with clobbers themselves).
template <int ACC>
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(ACC));
}

template <int ACC>
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "n"(ACC));
}

// Arrive on `bar` once every tcgen05.mma issued so far by this thread has completed.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 lanes x 32-bit, 16 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 32 lanes x 32-bit, 16 consecutive columns per thread, store.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Shared-memory matrix descriptor for a K-major (or MN-major) operand in the 128-byte swizzle
// layout: rows of 128 bytes, 8-row groups `sbo` bytes apart; `lbo` is the byte distance between
// 64-element column blocks for MN-major operands (ignored for K-major).  Layout-type 2 =
// SWIZZLE_128B, version 1 (sm_100).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t smem_addr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFF);
  d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFF) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version for sm_100
  d |= (uint64_t)2 << 61;  // SWIZZLE_128B
  return d;
}

// Descriptor for the no-swizzle ("interleaved") canonical layout: 8x16-byte core matrices,
// `lbo` bytes between core matrices adjacent in K, `sbo` bytes between 8-row groups.
__device__ __forceinline__ uint64_t noswz_desc(uint32_t smem_addr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFF);
  d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFF) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

// Instruction descriptor, kind::f16: f32 accumulate, A/B type (0 = f16, 1 = bf16), K-major A,
// B major as given, N and M dimensions.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t ab_type, uint32_t b_mn_major, uint32_t M,
                                                 uint32_t N) {
  return (1u << 4)                // D format f32
         | (ab_type << 7)         // A format
         | (ab_type << 10)        // B format
         | (0u << 15)             // A K-major
         | (b_mn_major << 16)     // B major
         | ((N >> 3) << 17)       // N / 8
         | ((M >> 4) << 24);      // M / 16
}

// Byte offset of the 16-byte chunk `chunk` (0..7) of row `r` inside a 128B-swizzled block whose
// rows are 128 bytes: chunks are XOR-permuted by the row index within each 8-row group.
__device__ __forceinline__ uint32_t sw128_offset(uint32_t r, uint32_t chunk) {
  return r * 128u + ((chunk ^ (r & 7u)) << 4);
}

}  // namespace dsa
