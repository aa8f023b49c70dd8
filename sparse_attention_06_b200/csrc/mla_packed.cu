// mla_packed.cu -- MLA over tiles of 128 query rows (mla_pair.cu has the kernel): how a call is planned and launched,
// the merging of key splits, and the expansion of quantised rows that several row tiles read.
//
// With several key splits per row tile each unit writes (O / l, LSE) partials that a small combine kernel merges:
// O = sum_sp exp(LSE_sp - LSE) O_sp, LSE = log sum_sp exp(LSE_sp).
#include "mla_packed.cuh"

namespace dsa {
namespace {

using namespace packed;

// grid (T, H), block 128: merge the split partials of one query row, out = sum_sp w_sp O_sp with
// w_sp = exp(LSE_sp - LSE); thread i sums the value columns 4 i .. 4 i + 3.
constexpr int kMaxSplits = 64;
template <bool kChunk>
__global__ void __launch_bounds__(128) combine_kernel(const Params p) {
  __shared__ float wts[kMaxSplits];
  __shared__ float s_inv, s_lse;
  const int t = blockIdx.x, h = blockIdx.y;
  griddep_launch_dependents();
  griddep_wait();
  int tile = t, r = h, n = p.nsplit;
  if constexpr (kChunk) {
    int req, pos;
    if (!chunk_token(p.chunks, t, &req, &pos, nullptr)) return;
    const int64_t flat = (int64_t)(t - p.chunks.cu_tokens[req]) * p.H + h;
    const int i = (int)(flat / kRows);
    r = (int)(flat % kRows);
    tile = (int)first_tile(p.chunks.cu_tokens[req], req, p.H) + i;
    int rows, row0, tok0, h0, len;
    if (!chunk_tile(p.chunks, p.H, req, i, rows, row0, tok0, h0, len, nullptr)) return;
    n = split_count(len, p.per);
    if (n == 1) return;  // written already
    const int tiles = (len + kTile - 1) / kTile, each = ((tiles + n - 1) / n + 1) / 2 * 2;
    n = (tiles + each - 1) / each;  // splits that have keys
  }
  const int64_t base = (int64_t)tile * p.nsplit * p.prows + r;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    float v[2], mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int sp = lane + 32 * e;
      v[e] = sp < n ? p.part_lse[base + (int64_t)sp * p.prows] : -INFINITY;
      mx = fmaxf(mx, v[e]);
    }
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      v[e] = v[e] == -INFINITY ? 0.0f : expf(v[e] - mx);
      wts[lane + 32 * e] = v[e];
      sum += v[e];
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) {
      s_inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      s_lse = sum == 0.0f ? -INFINITY : mx + logf(sum);
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float4* src = reinterpret_cast<const float4*>(p.part_o + base * kDv) + threadIdx.x;
  const int64_t step = (int64_t)p.prows * kDv / 4;
  for (int sp0 = 0; sp0 < n; sp0 += 16) {
    float4 a[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) a[e] = sp0 + e < n ? src[(sp0 + e) * step] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float w = sp0 + e < n ? wts[sp0 + e] : 0.0f;
      acc.x = fmaf(w, a[e].x, acc.x);
      acc.y = fmaf(w, a[e].y, acc.y);
      acc.z = fmaf(w, a[e].z, acc.z);
      acc.w = fmaf(w, a[e].w, acc.w);
    }
  }
  const float inv = s_inv;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 pk;
  pk.x = *reinterpret_cast<const uint32_t*>(&lo);
  pk.y = *reinterpret_cast<const uint32_t*>(&hi);
  const int64_t row = (int64_t)t * p.H + h;
  *reinterpret_cast<uint2*>(p.out + row * kDv + 4 * threadIdx.x) = pk;
  if (p.lse && threadIdx.x == 0) p.lse[row] = s_lse;
}

// Quantised rows of a batch of chunks as bf16 rows, once, for row tiles that would each turn them into bf16 again:
// a step of 128 keys costs the attention ~6000 cycles over quantised rows, ~4000 over bf16 ones.  One warp per position
// of a request that has tokens; rows[(request, position)], rows of pages outside the pool are left out (never read).
// Bound by memory: 15.5k rows (28 MB) in 9.4 us, cold.
constexpr int kExpandWarps = 4;
__global__ void __launch_bounds__(32 * kExpandWarps) expand_kernel(const uint8_t* data, const float* scale, int num_blocks,
                                                                   const dsa_chunks c, int linear_pages, __nv_bfloat16* rows,
                                                                   uint8_t* row_ok, int* err) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int per_req = linear_pages * kTile;
  const int64_t i = (int64_t)blockIdx.x * kExpandWarps + (threadIdx.x >> 5);
  const int r = (int)(i / per_req), pos = (int)(i % per_req);
  if (r >= c.num_reqs || pos >= c.max_context || pos >= c.seq_len[r] || c.cu_tokens[r + 1] <= c.cu_tokens[r]) return;
  const int32_t blk = c.block_table[(int64_t)r * c.max_blocks + pos / kTile];
  if (blk < 0 || blk >= num_blocks) return;
  const int64_t row = (int64_t)blk * kTile + pos % kTile;
  const uint8_t* src = data + row * kLatentBytes;
  uint2 w[2];
  float s[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = reinterpret_cast<const uint2*>(src + 256 * h)[lane];
    s[h] = scale[row * 4 + 2 * h + (lane >> 4)];
  }
  uint4 rope;
  if (lane < 8) rope = reinterpret_cast<const uint4*>(src + kDv)[lane];
  const bool ok = __all_sync(0xFFFFFFFFu, latent_scale_ok(s[0]) && latent_scale_ok(s[1]));
  if (lane == 0) {
    row_ok[i] = ok;
    if (!ok) raise_error(err, DSA_DEVERR_SCALE);
  }
  if (!ok) return;
  uint4* dst = reinterpret_cast<uint4*>(rows + i * kDqk);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t b[4];
    decode4(w[h].x, make_float2(s[h], s[h]), b[0], b[1]);
    decode4(w[h].y, make_float2(s[h], s[h]), b[2], b[3]);
    dst[32 * h + lane] = make_uint4(b[0], b[1], b[2], b[3]);
  }
  if (lane < 8) dst[64 + lane] = rope;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <Source kSrc>
cudaError_t launch(Params p, const MlaArgs& a, const void* data, int num_blocks, int num_sms, cudaStream_t s) {
  alignas(64) CUtensorMap qmap = {}, rmap = {}, pmap = {};
  if (!encode_tmap_2d(&qmap, a.q, 2, kDqk, (uint64_t)p.T * p.H, kDqk * 2, 64, kRows, true)) return cudaErrorInvalidValue;
  const uint64_t pool_rows = (uint64_t)num_blocks * kTile;  // of the rows that are copied
  // row numbers are 32-bit
  if (pool_rows >= 0x7FFFFFFFull || (int64_t)p.T * p.H + kRows >= 0x7FFFFFFFll ||
      (int64_t)p.tiles * p.nsplit * p.prows >= 0x7FFFFFFFll || (int64_t)p.tiles * p.nsplit * 2 >= 0x7FFFFFFFll)
    return cudaErrorInvalidValue;
  if (kSrc == kPagesBf16 && (!encode_tmap_2d(&rmap, data, 2, kDqk, pool_rows, kDqk * 2, 64, 1, true) ||
                             !encode_tmap_2d(&pmap, data, 2, kDqk, pool_rows, kDqk * 2, 64, kTile, true)))
    return cudaErrorInvalidValue;
  p.data = static_cast<const uint8_t*>(data);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.scale = a.latent.scale;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.oob_row = (int32_t)pool_rows;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.err = a.err;
  p.part_o = nullptr;
  p.part_lse = nullptr;
  if (p.nsplit > 1) {
    p.part_o = static_cast<float*>(a.workspace);
    p.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) +
                                          up256((size_t)p.tiles * p.nsplit * p.prows * kDv * sizeof(float)));
  }
  // several requests whose tiles are split: units differ in size, and are handed out as pairs become free.  (The counter
  // lives behind the partials; whole tiles go round robin, also where requests differ in length.)
  p.next = nullptr;
  if (kSrc != kSelected && p.nsplit > 1 && p.num_reqs > 1) {
    p.next = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(p.part_lse) + up256((size_t)p.tiles * p.nsplit * p.prows * sizeof(float)));
    const cudaError_t e = cudaMemsetAsync(p.next, 0, sizeof(int), s);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = launch_pair<kSrc>(p, qmap, rmap, pmap, num_sms, s);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  cudaLaunchAttribute cattrs[2];
  const cudaLaunchConfig_t ccfg = launch_config(dim3(p.T, p.H), dim3(128), 0, s, cattrs);
  return cudaLaunchKernelEx(&ccfg, combine_kernel<kSrc != kSelected>, p);
}

// Row tiles of a batch of chunks (an upper bound: the device knows the chunks' sizes).
int64_t chunk_tiles(int num_tokens, int num_reqs, int H) { return first_tile(num_tokens, num_reqs, H); }

}  // namespace

// Key tiles of a split of a batch of chunks, at most.  Cost model in the time of a 64-key tile (~1.3 us): a unit costs
// its key tiles and a fixed ~7 (queries in, output out); units are spread evenly over the SMs but for about half a unit
// at the end; several splits cost the combine's launch and the partials' way to memory and back.  Only max_context and
// the numbers of tokens and requests are known here; of several requests the mean length is taken as 0.6 of the
// longest.  (Measured: 7 requests of 71 to 308 tokens, 142 us in whole row tiles, 184 us in halves; 16 requests of 4
// tokens 182 and 181 us; one token at 2k context 19 us in 16 splits, 61 us whole in an earlier form.)
// Taking the mean as 1.0, 0.8, 0.6 or 0.4 of the longest, us, 128 heads, quantised: 16 requests of 4 tokens, all at 8000
// positions 302, 301, 226, 214; one at 16000 and the rest at 500 449, 156, 155, 256; half at 8000 and half at 500 178, 179,
// 154, 150; 32 requests of one token at 4000 93, 93, 101, 101, one at 16000 and the rest at 500 236, 236, 93, 136; two of 8
// tokens at 16000 and 100 92, 91, 67, 67.  Larger chunks (7 x 190 tokens of 16 heads, 4 x 300 of 128, 8 x 64 of 64) move by
// less than 3% but for one request of eight at 16000: 336, 275, 274, 278.
int chunk_mla_split_tiles(int num_tokens, int num_reqs, int H, int max_context, int num_sms) {
  // tiles in use if the tokens are spread evenly over the requests
  const int64_t per_req = ((int64_t)num_tokens * H + (int64_t)num_reqs * kRows - 1) / ((int64_t)num_reqs * kRows);
  const double tiles = (double)per_req * (num_reqs < num_tokens ? num_reqs : num_tokens);
  const double mean = num_reqs > 1 ? 0.6 : 1.0;
  const int kt = (max_context + kTile - 1) / kTile;
  double best_cost = 1e300;
  int best = kt;
  for (int n = 1; n <= kMaxSplits && n <= kt; n *= 2) {
    const int per = (kt + n - 1) / n;
    const double splits = mean * n > 1.0 ? mean * n : 1.0;
    const double units = 2.0 * tiles * splits;
    double cost = units <= num_sms ? per + 7.0 : 2.0 * tiles * (mean * kt + 7.0 * splits) / num_sms + 0.5 * (per + 7.0);
    if (n > 1) cost += 3.0 + 0.08 * tiles * splits;
    if (cost < best_cost) {
      best_cost = cost;
      best = per;
    }
  }
  return best;
}

namespace {
// Of a call with these sizes: the partials of split row tiles (and the unit counter), which it cannot do without, and
// the room for expanded rows, which it uses where there are quantised ones.
struct ChunkWorkspace {
  size_t partials, rows, total;
  int linear_pages;
};
ChunkWorkspace chunk_workspace(int num_tokens, int num_reqs, int H, int max_context, int split_tiles) {
  ChunkWorkspace w = {0, 0, 0, (max_context + kTile - 1) / kTile};
  const int nsplit = (w.linear_pages + split_tiles - 1) / split_tiles;
  if (nsplit > 1) {
    const size_t rows = (size_t)chunk_tiles(num_tokens, num_reqs, H) * nsplit * kRows;
    w.partials = up256(rows * kDv * sizeof(float)) + up256(rows * sizeof(float)) + 256;
  }
  // worth it from about three row tiles per request on (each 64-key tile then saves at least six CTAs ~1000 cycles for
  // ~3.5 MB/us of memory traffic spread over all SMs); bounded, since it grows with the contexts
  const size_t rows = (size_t)num_reqs * w.linear_pages * kTile;
  if ((int64_t)num_tokens * H > (int64_t)2 * kRows * num_reqs && rows * kDqk * 2 <= (256u << 20))
    w.rows = up256(rows * kDqk * 2) + up256(rows);
  w.total = w.partials + w.rows;
  return w;
}
}  // namespace

size_t chunk_mla_workspace(int num_tokens, int num_reqs, int H, int max_context, int split_tiles, bool least) {
  const ChunkWorkspace w = chunk_workspace(num_tokens, num_reqs, H, max_context, split_tiles);
  return least ? w.partials : w.total;
}

cudaError_t launch_chunk_mla_tc(const MlaArgs& a, const dsa_chunks& c, int split_tiles, int num_sms, cudaStream_t s, int* kernels) {
  Params p = {};
  p.chunks = c;
  p.block_table = c.block_table;
  p.T = c.num_tokens;
  p.H = a.H;
  p.per = split_tiles;
  p.cold = 1;
  p.nsplit = ((c.max_context + kTile - 1) / kTile + split_tiles - 1) / split_tiles;
  p.prows = kRows;
  const int64_t tiles = chunk_tiles(c.num_tokens, c.num_reqs, a.H);
  if (tiles >= 0x7FFFFFFFll) return cudaErrorInvalidValue;
  p.tiles = (int)tiles;
  p.num_reqs = c.num_reqs;
  p.max_blocks = c.max_blocks;
  p.max_context = c.max_context;
  const void* data = a.latent.data;
  const int blocks = a.latent.num_blocks;
  p.num_blocks = blocks;
  *kernels = p.nsplit > 1 ? 2 : 1;
  if (a.latent.dtype == DSA_BF16) return launch<kPagesBf16>(p, a, data, blocks, num_sms, s);
  const ChunkWorkspace w = chunk_workspace(c.num_tokens, c.num_reqs, a.H, c.max_context, split_tiles);
  if (!w.rows || a.workspace_bytes < w.total || (reinterpret_cast<uintptr_t>(a.workspace) & 255u)) return launch<kPages>(p, a, data, blocks, num_sms, s);
  const int64_t rows = (int64_t)c.num_reqs * w.linear_pages * kTile;
  uint8_t* at = static_cast<uint8_t*>(a.workspace) + w.partials;
  p.linear_pages = w.linear_pages;
  uint8_t* row_ok = at + up256((size_t)rows * kDqk * 2);
  p.row_ok = row_ok;
  cudaLaunchAttribute attrs[2];
  const cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)((rows + kExpandWarps - 1) / kExpandWarps)), dim3(32 * kExpandWarps), 0, s, attrs);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, expand_kernel, (const uint8_t*)data, a.latent.scale, blocks, c, w.linear_pages,
                                           reinterpret_cast<__nv_bfloat16*>(at), row_ok, a.err);
  if (e != cudaSuccess) return e;
  ++*kernels;
  return launch<kPagesBf16>(p, a, at, c.num_reqs * w.linear_pages, num_sms, s);
}

cudaError_t launch_mla_quantised_tc(const MlaArgs& a, int nsplit, int num_sms, cudaStream_t s) {
  Params p = {};
  p.idx = a.idx;
  p.q_req = a.batch.q_req;
  p.q_pos = a.batch.q_pos;
  p.block_table = a.batch.block_table;
  p.T = p.tiles = a.batch.num_queries;
  p.H = p.prows = a.H;
  p.k = a.k;
  // whole steps of 128 keys: at most the planned number of splits, whose partials the workspace holds
  p.ks = ((a.k + nsplit - 1) / nsplit + 2 * kTile - 1) / (2 * kTile) * (2 * kTile);
  p.nsplit = nsplit > 1 ? (a.k + p.ks - 1) / p.ks : 1;
  p.num_reqs = a.batch.num_reqs;
  p.max_blocks = a.batch.max_blocks;
  p.max_context = a.batch.max_context;
  p.num_blocks = a.latent.num_blocks;
  // Rows that several queries read are in L2 for all but the first: codes are fetched ahead where each row is read less
  // than twice on average.  (Decode of 64 queries at 16k context 76.4 us without, 73.2 with; 1024 queries of one
  // request 799 without, 825 with.)
  p.cold = (int64_t)a.batch.num_queries * a.k < 2 * (int64_t)a.batch.num_reqs * a.batch.max_context;
  return launch<kSelected>(p, a, a.latent.data, a.latent.num_blocks, num_sms, s);
}

}  // namespace dsa
