// cache.cu -- writing new tokens into the paged caches (quantising on the way) and reading rows back.
//
// Quantisation: a group of elements x gets the scale 2^e, e the smallest integer with
// max |x| <= 448 * 2^e (448 is the largest e4m3 value), and the codes RNE(x / 2^e).  With a
// power-of-two scale the division is exact, so a code is the correctly rounded x / 2^e, and
// code * 2^e has at most four significant bits: it is exact in bf16.  An arbitrary scale max|x| / 448
// would gain less than one binade of e4m3's subnormal end and lose both.
//
// Both directions move 656 + 1152 bytes per latent row and do a handful of operations per element:
// they are bound by HBM for many rows and by the chain of dependent loads (chunk bounds, block id,
// row) for few.  One warp per row: 16 codes a lane, so that a row's loads and stores are whole
// 512-byte runs and a 128-element group is eight lanes (three shuffles for its maximum).
#include "common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kWarps = 8;
constexpr int kLatent = 512, kRope = 64, kLatentRowBytes = kLatent + 2 * kRope;

// Pool row of position `pos` of request `req`, -1 (flagged) when its block id is outside the pool.
__device__ __forceinline__ int64_t pool_row(const dsa_chunks& c, const dsa_paged_cache& cache, int req, int pos, int* err) {
  const int32_t blk = c.block_table[(int64_t)req * c.max_blocks + pos / 64];
  if (blk < 0 || blk >= cache.num_blocks) {
    raise_error(err, DSA_DEVERR_BLOCK_ID);
    return -1;
  }
  return (int64_t)blk * 64 + pos % 64;
}

// Exponent e of a group's scale 2^e from its largest finite magnitude (bits of a float >= 0):
// 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - ((b & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  return amax == 0.0f ? 0 : max(-100, min(119, e));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// NaN for an infinity or NaN; `bad` notes it.
__device__ __forceinline__ float finite_or_nan(float x, bool& bad) {
  if (fabsf(x) <= 3.402823466e38f) return x;
  bad = true;
  return __uint_as_float(0x7FC00000u);
}
// fmaxf ignores NaN, so the group maximum is over the finite elements
__device__ __forceinline__ float amax_step(float m, float x) { return fmaxf(m, fabsf(x)); }

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// N consecutive elements (8-byte multiples) from x + i, as f32
template <int N>
__device__ __forceinline__ void load_elems(const void* x, int dtype, int64_t i, float (&v)[N]) {
  if (dtype == DSA_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(x) + i;
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int e = 0; e < N / 8; ++e) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + e);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * e + 2 * j] = __uint_as_float(u[j] << 16);
          v[8 * e + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p) + e);
        v[2 * e] = __uint_as_float(w << 16);
        v[2 * e + 1] = __uint_as_float(w & 0xFFFF0000u);
      }
    }
  } else {
    const float* p = static_cast<const float*>(x) + i;
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int e = 0; e < N / 4; ++e) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(p) + e);
        v[4 * e] = w.x; v[4 * e + 1] = w.y; v[4 * e + 2] = w.z; v[4 * e + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const float2 w = __ldg(reinterpret_cast<const float2*>(p) + e);
        v[2 * e] = w.x; v[2 * e + 1] = w.y;
      }
    }
  }
}

// One group of `n` elements by a warp, any n and alignment: the plain path.
__device__ void quantise_any(const void* x, int dtype, int64_t i0, int n, uint8_t* codes, float* scale, bool& bad) {
  const int lane = threadIdx.x & 31;
  float m = 0.0f;
  bool b = false;
  for (int i = lane; i < n; i += 32) m = amax_step(m, finite_or_nan(load_elem(x, dtype, i0 + i), b));
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const int e = scale_exponent(m);
  const float inv = pow2(-e);
  for (int i = lane; i < n; i += 32)
    codes[i] = (uint8_t)__nv_cvt_float_to_fp8(finite_or_nan(load_elem(x, dtype, i0 + i), b) * inv, __NV_SATFINITE, __NV_E4M3);
  if (lane == 0) *scale = pow2(e);
  bad |= b;
}

// A row of n elements into an unquantised cache.
__device__ void copy_any(const void* x, int x_dtype, int64_t i0, int n, void* dst, int dst_dtype, int64_t o0) {
  for (int i = threadIdx.x & 31; i < n; i += 32) {
    const float v = load_elem(x, x_dtype, i0 + i);
    if (dst_dtype == DSA_F32)
      static_cast<float*>(dst)[o0 + i] = v;
    else
      static_cast<__nv_bfloat16*>(dst)[o0 + i] = __float2bfloat16_rn(v);
  }
}

// kFast: every quantised input row starts on a 16-byte boundary (and keys, if quantised, have 128
// elements), so rows move as vectors; else element by element.
template <bool kFast>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  int req, pos;
  if (!chunk_token(a.chunks, t, &req, &pos, lane == 0 ? a.err : nullptr)) return;
  bool bad = false;
  if (a.k) {
    const int64_t row = pool_row(a.chunks, a.keys, req, pos, lane == 0 ? a.err : nullptr);
    const int n = a.keys.dim;
    const int64_t i0 = (int64_t)t * a.k_stride;
    if (row >= 0) {
      if (a.keys.dtype != DSA_E4M3) {
        copy_any(a.k, a.x_dtype, i0, n, const_cast<void*>(a.keys.data), a.keys.dtype, row * n);
      } else {
        uint8_t* codes = static_cast<uint8_t*>(const_cast<void*>(a.keys.data)) + row * n;
        float* scale = const_cast<float*>(a.keys.scale) + row;
        if constexpr (kFast) {
          float v[4];
          load_elems(a.k, a.x_dtype, i0 + 4 * lane, v);
          float m = 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) m = amax_step(m, v[j] = finite_or_nan(v[j], bad));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          const int e = scale_exponent(m);
          const float inv = pow2(-e);
          reinterpret_cast<uint32_t*>(codes)[lane] = pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
          if (lane == 0) *scale = pow2(e);
        } else {
          quantise_any(a.k, a.x_dtype, i0, n, codes, scale, bad);
        }
      }
    }
  }
  if (a.kv) {
    const int64_t row = pool_row(a.chunks, a.latent, req, pos, lane == 0 ? a.err : nullptr);
    const int n = a.latent.dim;
    const int64_t i0 = (int64_t)t * a.kv_stride;
    if (row >= 0) {
      if (a.latent.dtype != DSA_LATENT_E4M3) {
        copy_any(a.kv, a.x_dtype, i0, n, const_cast<void*>(a.latent.data), a.latent.dtype, row * n);
      } else {
        uint8_t* codes = static_cast<uint8_t*>(const_cast<void*>(a.latent.data)) + row * kLatentRowBytes;
        float* scale = const_cast<float*>(a.latent.scale) + row * 4;
        if constexpr (kFast) {
          float v[16];  // elements 16 lane .. 16 lane + 15: eight lanes are one group of 128
          load_elems(a.kv, a.x_dtype, i0 + 16 * lane, v);
          float rope[2];
          load_elems(a.kv, a.x_dtype, i0 + kLatent + 2 * lane, rope);
          float m = 0.0f;
#pragma unroll
          for (int j = 0; j < 16; ++j) m = amax_step(m, v[j] = finite_or_nan(v[j], bad));
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          const int e = scale_exponent(m);
          const float inv = pow2(-e);
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = pack4(v[4 * j] * inv, v[4 * j + 1] * inv, v[4 * j + 2] * inv, v[4 * j + 3] * inv);
          reinterpret_cast<uint4*>(codes)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
          const __nv_bfloat162 r2 = __floats2bfloat162_rn(rope[0], rope[1]);
          reinterpret_cast<__nv_bfloat162*>(codes + kLatent)[lane] = r2;
          if ((lane & 7) == 0) scale[lane >> 3] = pow2(e);
        } else {
          for (int g = 0; g < kLatent / 128; ++g) quantise_any(a.kv, a.x_dtype, i0 + 128 * g, 128, codes + 128 * g, scale + g, bad);
          copy_any(a.kv, a.x_dtype, i0 + kLatent, kRope, codes + kLatent, DSA_BF16, 0);
        }
      }
    }
  }
  if (bad) raise_error(a.err, DSA_DEVERR_NONFINITE);
}

__device__ __forceinline__ void store_elem(void* out, int dtype, int64_t i, float v) {
  if (dtype == DSA_F32)
    static_cast<float*>(out)[i] = v;
  else
    static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

__global__ void __launch_bounds__(32 * kWarps) read_kernel(const ReadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  int req, pos;
  if (!chunk_token(a.chunks, t, &req, &pos, lane == 0 ? a.err : nullptr)) return;
  const int64_t row = pool_row(a.chunks, a.cache, req, pos, lane == 0 ? a.err : nullptr);
  if (row < 0) return;
  const int n = a.cache.dim;
  for (int i = lane; i < n; i += 32) store_elem(a.out, a.out_dtype, (int64_t)t * n + i, load_cached(a.cache, row, i));
}

bool aligned(const void* p, int64_t stride_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes) & 15u) == 0;
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  const int64_t size = a.x_dtype == DSA_BF16 ? 2 : 4;
  const bool k_ok = !a.k || a.keys.dtype != DSA_E4M3 || (a.keys.dim == 128 && aligned(a.k, a.k_stride * size));
  const bool kv_ok = !a.kv || a.latent.dtype != DSA_LATENT_E4M3 || aligned(a.kv, a.kv_stride * size);
  cudaLaunchAttribute attrs[2];
  const cudaLaunchConfig_t cfg =
      launch_config(dim3((a.chunks.num_tokens + kWarps - 1) / kWarps), dim3(32 * kWarps), 0, s, attrs);
  return cudaLaunchKernelEx(&cfg, k_ok && kv_ok ? append_kernel<true> : append_kernel<false>, a);
}

cudaError_t launch_cache_read(const ReadArgs& a, cudaStream_t s) {
  cudaLaunchAttribute attrs[2];
  const cudaLaunchConfig_t cfg =
      launch_config(dim3((a.chunks.num_tokens + kWarps - 1) / kWarps), dim3(32 * kWarps), 0, s, attrs);
  return cudaLaunchKernelEx(&cfg, read_kernel, a);
}

}  // namespace dsa
