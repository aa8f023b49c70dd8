// mla_packed.cuh -- what the MLA kernels over tiles of 128 query rows share: the tile's shape, the units of
// work and how a batch of chunks is cut into them, arithmetic, the epilogue's store.
#pragma once

#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "mla_pair_layout.h"

namespace dsa {
namespace packed {

constexpr int kLatentBytes = 640;        // data bytes of a quantised row

__device__ __forceinline__ int block_of(int pos, int v) {  // column block of a row at place `pos` of that order
  return pos == 0 ? 8 : pos < 5 ? 4 * (1 - v) + (pos == 1 ? 3 : pos - 2) : 4 * v + pos - 5;
}

constexpr uint32_t TM_O = 0, TM_S = 256, TM_Q = 320, TM_COLS = 512;

// Where a unit's keys come from.
enum Source {
  kSelected,   // quantised rows chosen per query by idx (or every visible position)
  kPages,      // quantised rows at consecutive positions
  kPagesBf16,  // bf16 rows at consecutive positions
};

struct Params {
  const uint8_t* data;    // pool rows
  const __nv_bfloat16* q;  // [T, H, 576]
  const float* scale;     // quantised: [pool rows, 4]
  const int32_t* idx;     // kSelected: [T, k] or null (every visible position)
  const int32_t *q_req, *q_pos;
  dsa_chunks chunks;      // kPages*
  const int32_t* block_table;
  __nv_bfloat16* out;     // [T, H, 512]
  float* lse;             // [T, H] or null
  float *part_o, *part_lse;  // several splits: [tiles, nsplit, prows, 512] and [tiles, nsplit, prows]
  const uint8_t* row_ok;  // kPagesBf16 over expanded rows: [requests, linear_pages * 64] rows with good scales
  int linear_pages;       // ... whose pages follow each other, so many for each request; 0: pages of the pool
  int32_t num_blocks, oob_row;
  int T, H, k, ks, nsplit, per, prows, tiles, num_reqs, max_blocks, max_context;
  int* next;              // units handed out beyond the first of each CTA pair (zero at launch), or null: round robin
  int cold;               // quantised rows are probably not in L2
  float scale_log2;       // softmax scale * log2(e)
  int* err;
};

// A unit of work.
struct Unit {
  int rows;       // query rows in use; 0: nothing to do, -1: no more units
  int row0;       // first of them in the [T * H] query rows
  int req;        // request (-1: the query is invalid, it sees nothing)
  int tok0, h0;   // kPages*: token of row 0 within its chunk's positions (its position), its head
  int lo, hi;     // keys: selection slots or positions [lo, hi)
  int splits;     // of the row tile: 1 writes the output, more write partials
  int prow;       // first partial row
  int v;
};
static_assert(sizeof(Unit) == kUnitBytes, "unit ring");

template <bool B>
struct Flag {
  static constexpr bool value = B;
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // relative error ~2^-22; 2^-inf = 0
  return y;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// 16-byte cp.async past L1; bytes from `size` (0 or 16) on are zeros
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}

// Loads that stay where they are written: left to itself the compiler moves loads for later down to their use, and
// with them their whole latency.  (Not the non-coherent path: the kernel that writes the rows may end after this one began.)
__device__ __forceinline__ uint4 load16_here(const void* a) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(a));
  return v;
}
__device__ __forceinline__ float loadf_here(const float* a) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(a));
  return v;
}

// two f32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Tiles of a batch of chunks: request r has the tile numbers first_tile(r) .. first_tile(r + 1) - 1, at
// least as many as its rows need (ceil(b - a) <= floor(b) - floor(a) + 1); the rest are unused.  So a
// tile's request follows from cu_tokens alone, by a search instead of a prefix sum.
__host__ __device__ __forceinline__ int64_t first_tile(int64_t cu, int r, int H) { return cu * H / kRows + r; }

// Request of tile `tile` (warp-collective): a 32-way search of the last r with first_tile(r) <= tile;
// -1 when there is none.
__device__ __forceinline__ int tile_request(const dsa_chunks& c, int H, int tile) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = c.num_reqs;  // candidates lo .. lo + n - 1
  while (true) {
    const int step = (n + 31) / 32;
    const int r = lo + lane * step;
    const bool le = lane * step < n && first_tile(max(0, c.cu_tokens[r]), r, H) <= tile;
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, le);
    if (b == 0u) return -1;
    const int last = 31 - __clz(b);
    lo += last * step;
    n = min(step, n - last * step);
    if (step == 1) return lo;
  }
}

// Key splits of a row tile that sees positions 0 .. len - 1: as many as it takes for at most `per` key tiles each
// (units of like size keep the CTAs busy to the end, however ragged the batch), and split sp's keys: pairs of
// key tiles, evenly.
__device__ __forceinline__ int split_count(int len, int per) { return ((len + kTile - 1) / kTile + per - 1) / per; }
__device__ __forceinline__ void split_range(int len, int splits, int sp, int& lo, int& hi) {
  const int tiles = (len + kTile - 1) / kTile, each = ((tiles + splits - 1) / splits + 1) / 2 * 2;
  lo = min(len, sp * each * kTile);
  hi = min(len, lo + each * kTile);
}

// Row tile `i` of request r: its rows, the position of its first and behind its last token.
__device__ __forceinline__ bool chunk_tile(const dsa_chunks& c, int H, int r, int i, int& rows, int& row0, int& tok0, int& h0,
                                           int& len, int* err) {
  const int first = c.cu_tokens[r], end = c.cu_tokens[r + 1], seq = c.seq_len[r];
  if (first == end) return false;
  if (first < 0 || end < first || end > c.num_tokens || seq > c.max_context || seq < end - first) {
    raise_error(err, DSA_DEVERR_REQUEST);
    return false;
  }
  const int64_t all = (int64_t)(end - first) * H, f = (int64_t)i * kRows;
  if (f >= all) return false;
  rows = (int)min((int64_t)kRows, all - f);
  row0 = (int)((int64_t)first * H + f);
  const int ctx = seq - (end - first);
  tok0 = ctx + (int)(f / H);
  h0 = (int)(f % H);
  len = ctx + (int)((f + rows - 1) / H) + 1;
  return true;
}

// Unit u, by a whole warp.  Chunks: late tiles first (they see the most keys of a prompt).
template <Source kSrc>
__device__ __forceinline__ Unit get_unit(const Params& p, int u, int* err) {
  Unit x;
  x.rows = 0;
  x.v = u & 1;
  x.splits = p.nsplit;
  const int ts = u >> 1;
  const int sp = ts % p.nsplit;
  int tile = ts / p.nsplit;
  if constexpr (kSrc == kSelected) {
    x.rows = p.H;
    x.row0 = tile * p.H;
    x.req = p.q_req[tile];
    x.tok0 = p.q_pos[tile];
    x.h0 = 0;
    if (x.req < 0 || x.req >= p.num_reqs || x.tok0 < 0 || x.tok0 >= p.max_context) {
      raise_error(err, DSA_DEVERR_REQUEST);
      x.req = -1;
    }
    const int slots = p.idx ? p.k : (x.req < 0 ? 0 : min(p.k, x.tok0 + 1));
    x.lo = min(slots, sp * p.ks);
    x.hi = min(slots, x.lo + p.ks);
  } else {
    tile = p.tiles - 1 - tile;
    const int r = tile_request(p.chunks, p.H, tile);
    if (r < 0) return x;
    int len;
    const int i = tile - (int)first_tile(max(0, p.chunks.cu_tokens[r]), r, p.H);
    if (!chunk_tile(p.chunks, p.H, r, i, x.rows, x.row0, x.tok0, x.h0, len, err)) {
      x.rows = 0;
      return x;
    }
    x.req = r;
    x.splits = split_count(len, p.per);
    split_range(len, x.splits, sp, x.lo, x.hi);
    if (sp >= x.splits || x.lo >= x.hi) x.rows = 0;  // (a split without keys leaves no partial: the combine knows it)
  }
  x.prow = (tile * p.nsplit + sp) * p.prows;
  return x;
}

// Four codes times their scale as two bf16 pairs, all exact (four significant bits and a power of two): the
// hardware's e4m3 -> f16 conversion, f32 products, one packing conversion.  Of the ten instructions four are ALU ones;
// moving the code's bits into a bf16's with integer operations took thirteen, eleven of them ALU, whose
// half-rate pipe then bounds the kernel.
__device__ __forceinline__ void decode4(uint32_t w, float2 s, uint32_t& lo, uint32_t& hi) {
  uint32_t h[2], b[2];
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = mul2(__half22float2(*reinterpret_cast<const __half2*>(&h[i])), s);
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x, f.y);
    b[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  lo = b[0];
  hi = b[1];
}

// O_v / l of this warp's 32 rows, columns [c_lo, c_hi) (multiples of 32), from tensor memory to the
// partials (f32) or the output (bf16) through a 2 KB staging area of its own: lane i stages 64 bytes of its row, its
// 16-byte pieces permuted against bank conflicts, then the warp writes whole 64-byte pieces of eight rows at a time.
__device__ __forceinline__ void store_o(const Params& p, const Unit& x, uint32_t lane_base, int quarter, int c_lo, int c_hi,
                                        uint8_t* stage, float inv, bool have_o) {
  const int lane = threadIdx.x & 31;
  const bool f32out = x.splits > 1;
  const int rows = min(32, x.rows - quarter * 32);
  uint8_t* mine = stage + lane * 64;
  const int mix = (lane >> 1) & 3;
  auto flush = [&](int col) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int rr = k * 8 + (lane >> 2), piece = lane & 3;
      const uint4 y = *reinterpret_cast<const uint4*>(stage + rr * 64 + ((piece ^ ((rr >> 1) & 3)) << 4));
      if (rr < rows) {
        if (f32out)
          *reinterpret_cast<uint4*>(p.part_o + ((int64_t)x.prow + quarter * 32 + rr) * kDv + x.v * kHalf + col + piece * 4) = y;
        else
          *reinterpret_cast<uint4*>(p.out + ((int64_t)x.row0 + quarter * 32 + rr) * kDv + x.v * kHalf + col + piece * 8) = y;
      }
    }
    __syncwarp();
  };
  if (rows <= 0) return;
#pragma unroll 1
  for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
    uint32_t o[32];
    if (have_o) {
#pragma unroll
      for (int c = 0; c < 2; ++c) tmem_ld16(lane_base + TM_O + c0 + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&o[16 * c]));
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) o[c] = 0u;
    }
    if (f32out) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = 16 * b + 4 * j;
          *reinterpret_cast<float4*>(mine + ((j ^ mix) << 4)) =
              make_float4(__uint_as_float(o[c]) * inv, __uint_as_float(o[c + 1]) * inv, __uint_as_float(o[c + 2]) * inv,
                          __uint_as_float(o[c + 3]) * inv);
        }
        flush(c0 + 16 * b);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t pk[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 hv =
              __floats2bfloat162_rn(__uint_as_float(o[8 * j + 2 * e]) * inv, __uint_as_float(o[8 * j + 2 * e + 1]) * inv);
          pk[e] = *reinterpret_cast<const uint32_t*>(&hv);
        }
        *reinterpret_cast<uint4*>(mine + ((j ^ mix) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
      flush(c0);
    }
  }
}

// The kernel on CTA pairs (mla_pair.cu), for every source: tensor maps of the queries (128-row boxes) and, of bf16 rows, of
// the rows one by one and of whole pages.
template <Source kSrc>
cudaError_t launch_pair(const Params& p, const CUtensorMap& qmap, const CUtensorMap& rmap, const CUtensorMap& pmap, int num_sms,
                        cudaStream_t s);

}  // namespace packed
}  // namespace dsa
