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
// row) for few.  One warp per row; writing, its input is on the way before the row is looked up.  A row
// goes in pieces of eight elements, one per lane, so that loads and stores are whole runs of 256 or
// 512 bytes; a 128-element group is sixteen lanes (four shuffles for its maximum).
//
// A kernel here may begin before the one that writes its inputs or rows has ended (griddepcontrol), so these are read with
// ordinary loads: the non-coherent path is for memory that nobody writes while the kernel lives.  (Both measured: reads
// of 281k rows alike, 85 us; appends of as many 139 -> 132 us into quantised caches, 162 -> 146 into bf16 ones.)
#include "common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kWarps = 4;  // of a block, one token each
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
        const uint4 w = reinterpret_cast<const uint4*>(p)[e];
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
        const uint32_t w = reinterpret_cast<const uint32_t*>(p)[e];
        v[2 * e] = __uint_as_float(w << 16);
        v[2 * e + 1] = __uint_as_float(w & 0xFFFF0000u);
      }
    }
  } else {
    const float* p = static_cast<const float*>(x) + i;
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int e = 0; e < N / 4; ++e) {
        const float4 w = reinterpret_cast<const float4*>(p)[e];
        v[4 * e] = w.x; v[4 * e + 1] = w.y; v[4 * e + 2] = w.z; v[4 * e + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const float2 w = reinterpret_cast<const float2*>(p)[e];
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

// Request of token t (warp-collective, the same t in every lane): the last r with cu_tokens[r] <= t, by a 32-way
// search (two rounds of loads for a thousand requests); t lies within cu_tokens[0] .. cu_tokens[num_reqs] - 1.
__device__ __forceinline__ int find_request(const dsa_chunks& c, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = c.num_reqs;
  while (true) {
    const int step = (n + 31) / 32;
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, lane * step < n && c.cu_tokens[lo + lane * step] <= t) | 1u;
    const int last = 31 - __clz(b);
    lo += last * step;
    n = min(step, n - last * step);
    if (step == 1) return lo;
  }
}

// Request and position of token t (warp-collective); false for a row that is no request's, and for one whose
// request has bounds outside the call's (flagged).
__device__ __forceinline__ bool find_token(const dsa_chunks& c, int t, int* req, int* pos, int* err) {
  if (t < c.cu_tokens[0] || t >= c.cu_tokens[c.num_reqs]) return false;
  const int r = find_request(c, t);
  const int first = c.cu_tokens[r], end = c.cu_tokens[r + 1], len = c.seq_len[r];
  if (first < 0 || end > c.num_tokens || len > c.max_context || len < end - first) {
    if ((threadIdx.x & 31) == 0) raise_error(err, DSA_DEVERR_REQUEST);
    return false;
  }
  *req = r;
  *pos = len - (end - t);
  return true;
}

__device__ __forceinline__ void store8(void* out, int dtype, int64_t i, const float (&v)[8]) {
  if (dtype == DSA_F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + i);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A row of n elements (a multiple of 8, both sides on 16 bytes) into an unquantised cache.
__device__ __forceinline__ void copy_row(const void* x, int x_dtype, int64_t i0, const dsa_paged_cache& c, int64_t row) {
  for (int i = 8 * (threadIdx.x & 31); i < c.dim; i += 256) {
    float v[8];
    load_elems(x, x_dtype, i0 + i, v);
    store8(const_cast<void*>(c.data), c.dtype, row * c.dim + i, v);
  }
}

// Eight consecutive elements as they are in memory (registers are what bounds the warps in flight).
template <bool kBf16>
struct Raw8 {
  uint4 w[kBf16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* x, int64_t i) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + i * (kBf16 ? 2 : 4));
#pragma unroll
    for (int e = 0; e < (kBf16 ? 1 : 2); ++e) w[e] = p[e];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[kBf16 ? 0 : 1].x, w[kBf16 ? 0 : 1].y, w[kBf16 ? 0 : 1].z, w[kBf16 ? 0 : 1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(kBf16 ? (j & 1 ? u[j >> 1] & 0xFFFF0000u : u[j >> 1] << 16) : u[j]);
  }
  // bits of the largest magnitude, as f32
  __device__ __forceinline__ uint32_t absmax_bits() const {
    if constexpr (kBf16) {
      const uint32_t k = 0x7FFF7FFFu;
      const uint32_t m = __vmaxu2(__vmaxu2(w[0].x & k, w[0].y & k), __vmaxu2(w[0].z & k, w[0].w & k));
      return max(m & 0xFFFF0000u, m << 16);
    } else {
      const uint32_t k = 0x7FFFFFFFu;
      return max(max(max(w[0].x & k, w[0].y & k), max(w[0].z & k, w[0].w & k)),
                 max(max(w[1].x & k, w[1].y & k), max(w[1].z & k, w[1].w & k)));
    }
  }
};

// Eight elements of a 128-element group that sixteen neighbouring lanes hold: codes, and the group's scale.
// Magnitudes are compared as integers (the bits of |x| are in the order of |x|, infinities and NaN on top), so
// that only a group with one of those looks at its elements one by one.
template <bool kBf16>
__device__ __forceinline__ uint2 quantise8(const Raw8<kBf16>& x, float* scale, bool& bad) {
  uint32_t m = x.absmax_bits();
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float v[8];
  x.get(v);
  if (m >= 0x7F800000u) {
    float f = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f = amax_step(f, v[j] = finite_or_nan(v[j], bad));
    const uint32_t half = 0xFFFFu << (threadIdx.x & 16);  // (the group's lanes took this branch together)
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) f = fmaxf(f, __shfl_xor_sync(half, f, o));
    m = __float_as_uint(f);
  }
  const int e = scale_exponent(__uint_as_float(m));
  const float inv = pow2(-e);
  *scale = pow2(e);
  return make_uint2(pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv), pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// One warp per token.  kFast: rows of the inputs start on 16 bytes, their widths are multiples of 8 and
// quantised keys have 128 elements; else element by element.  kBf16: type of the inputs (kFast).
// Measured: 64 tokens in 2.8 us (launch), 13k tokens into both quantised caches (28 MB) in 7.7 us, 3.6 TB/s.
template <bool kFast, bool kBf16>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.chunks.num_tokens) return;
  const int64_t k0 = (int64_t)t * a.k_stride, v0 = (int64_t)t * a.kv_stride;
  const bool qk = kFast && a.k && a.keys.dtype == DSA_E4M3, qv = kFast && a.kv && a.latent.dtype == DSA_LATENT_E4M3;
  // the inputs are on their way while the row is looked up
  Raw8<kBf16> v[2], kk;
  float rope[2];
  if (qv) {
    v[0].load(a.kv, v0 + 8 * lane);
    v[1].load(a.kv, v0 + 256 + 8 * lane);
    load_elems(a.kv, a.x_dtype, v0 + kLatent + 2 * lane, rope);
  }
  if (qk) kk.load(a.k, k0 + 8 * (lane & 15));
  int req, pos;
  if (!find_token(a.chunks, t, &req, &pos, a.err)) return;
  int* lane_err = lane == 0 ? a.err : nullptr;
  const int64_t kr = a.k ? pool_row(a.chunks, a.keys, req, pos, lane_err) : -1;
  const int64_t vr = a.kv ? pool_row(a.chunks, a.latent, req, pos, lane_err) : -1;
  bool bad = false;
  if (vr >= 0) {
    if (a.latent.dtype == DSA_LATENT_E4M3) {
      uint8_t* codes = static_cast<uint8_t*>(const_cast<void*>(a.latent.data)) + vr * kLatentRowBytes;
      float* scale = const_cast<float*>(a.latent.scale) + vr * 4;
      if (kFast) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float s;
          reinterpret_cast<uint2*>(codes + 256 * h)[lane] = quantise8(v[h], &s, bad);
          if ((lane & 15) == 0) scale[2 * h + (lane >> 4)] = s;
        }
        reinterpret_cast<__nv_bfloat162*>(codes + kLatent)[lane] = __floats2bfloat162_rn(rope[0], rope[1]);
      } else {
        for (int g = 0; g < kLatent / 128; ++g) quantise_any(a.kv, a.x_dtype, v0 + 128 * g, 128, codes + 128 * g, scale + g, bad);
        copy_any(a.kv, a.x_dtype, v0 + kLatent, kRope, codes + kLatent, DSA_BF16, 0);
      }
    } else if (kFast) {
      copy_row(a.kv, a.x_dtype, v0, a.latent, vr);
    } else {
      copy_any(a.kv, a.x_dtype, v0, a.latent.dim, const_cast<void*>(a.latent.data), a.latent.dtype, vr * a.latent.dim);
    }
  }
  if (kr >= 0) {
    const int n = a.keys.dim;
    uint8_t* codes = static_cast<uint8_t*>(const_cast<void*>(a.keys.data)) + kr * n;
    float* scale = const_cast<float*>(a.keys.scale) + kr;
    if (a.keys.dtype == DSA_E4M3) {
      if (kFast) {
        float s;
        const uint2 w = quantise8(kk, &s, bad);  // (the upper sixteen lanes repeat the lower)
        if (lane < 16) reinterpret_cast<uint2*>(codes)[lane] = w;
        if (lane == 0) *scale = s;
      } else {
        quantise_any(a.k, a.x_dtype, k0, n, codes, scale, bad);
      }
    } else if (kFast) {
      copy_row(a.k, a.x_dtype, k0, a.keys, kr);
    } else {
      copy_any(a.k, a.x_dtype, k0, n, const_cast<void*>(a.keys.data), a.keys.dtype, kr * n);
    }
  }
  if (bad) raise_error(a.err, DSA_DEVERR_NONFINITE);
}

// Eight codes times a scale (exact for a power of two).
__device__ __forceinline__ void decode8(uint2 w, float s, float (&v)[8]) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

__device__ __forceinline__ void store_elem(void* out, int dtype, int64_t i, float v) {
  if (dtype == DSA_F32)
    static_cast<float*>(out)[i] = v;
  else
    static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

// One warp per token.  kFast: out on 16 bytes and rows of a multiple of 8 elements; else element by element.
// Measured: 281k quantised rows to bf16 (513 MB) in 87 us, 5.9 TB/s; two rows a warp 91 us, four 109 us (their
// registers cost more warps than their loads in flight are worth).
template <bool kFast>
__global__ void __launch_bounds__(32 * kWarps) read_kernel(const ReadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  int req, pos;
  if (t >= a.chunks.num_tokens || !find_token(a.chunks, t, &req, &pos, a.err)) return;
  const int64_t row = pool_row(a.chunks, a.cache, req, pos, lane == 0 ? a.err : nullptr);
  if (row < 0) return;
  const int n = a.cache.dim;
  const int64_t o = (int64_t)t * n;
  const uint8_t* data = static_cast<const uint8_t*>(a.cache.data);
  if constexpr (!kFast) {
    for (int i = lane; i < n; i += 32) store_elem(a.out, a.out_dtype, o + i, load_cached(a.cache, row, i));
  } else if (a.cache.dtype == DSA_LATENT_E4M3) {
    const uint8_t* src = data + row * kLatentRowBytes;
    uint2 w[2];
    float s[2], rope[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = reinterpret_cast<const uint2*>(src + 256 * h)[lane];
      s[h] = a.cache.scale[row * 4 + 2 * h + (lane >> 4)];
    }
    if (lane < 8) load_elems(src + kLatent, DSA_BF16, 8 * lane, rope);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
      decode8(w[h], s[h], v);
      store8(a.out, a.out_dtype, o + 256 * h + 8 * lane, v);
    }
    if (lane < 8) store8(a.out, a.out_dtype, o + kLatent + 8 * lane, rope);
  } else if (a.cache.dtype == DSA_E4M3) {
    for (int i = 8 * lane; i < n; i += 256) {
      const uint2 w = *reinterpret_cast<const uint2*>(data + row * n + i);
      float v[8];
      decode8(w, a.cache.scale[row], v);
      store8(a.out, a.out_dtype, o + i, v);
    }
  } else {
    for (int i = 8 * lane; i < n; i += 256) {
      float v[8];
      load_elems(data, a.cache.dtype, row * n + i, v);
      store8(a.out, a.out_dtype, o + i, v);
    }
  }
}

bool on16(const void* p, int64_t row_bytes) { return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)row_bytes) & 15u) == 0; }

unsigned blocks(int tokens, int per_block) { return ((unsigned)tokens + per_block - 1) / per_block; }

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  const int64_t size = a.x_dtype == DSA_BF16 ? 2 : 4;
  const bool k_ok = !a.k || (on16(a.k, a.k_stride * size) && a.keys.dim % 8 == 0 && (a.keys.dtype != DSA_E4M3 || a.keys.dim == 128));
  const bool kv_ok = !a.kv || (on16(a.kv, a.kv_stride * size) && a.latent.dim % 8 == 0);
  cudaLaunchAttribute attrs[2];
  const cudaLaunchConfig_t cfg = launch_config(dim3(blocks(a.chunks.num_tokens, kWarps)), dim3(32 * kWarps), 0, s, attrs);
  const bool fast = k_ok && kv_ok;
  return cudaLaunchKernelEx(&cfg, !fast ? append_kernel<false, true> : a.x_dtype == DSA_BF16 ? append_kernel<true, true> : append_kernel<true, false>, a);
}

cudaError_t launch_cache_read(const ReadArgs& a, cudaStream_t s) {
  cudaLaunchAttribute attrs[2];
  const cudaLaunchConfig_t cfg = launch_config(dim3(blocks(a.chunks.num_tokens, kWarps)), dim3(32 * kWarps), 0, s, attrs);
  const bool fast = on16(a.out, 0) && a.cache.dim % 8 == 0;
  return cudaLaunchKernelEx(&cfg, fast ? read_kernel<true> : read_kernel<false>, a);
}

}  // namespace dsa
