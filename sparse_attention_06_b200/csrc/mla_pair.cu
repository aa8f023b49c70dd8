// mla_pair.cu -- MLA (MQA mode) for tiles of 128 query rows on tcgen05 tensor cores, a CTA pair to a tile: dense
// attention of chunks over the paged latent cache, and sparse attention over quantised latents.
//
// Mathematics: out = softmax(tau Q K^T + mask) V with K the 576-wide latent rows and V their first 512 elements, by
// one pass over the keys with a running maximum and sum per query row.
//
// Query rows.  A token's H heads are H rows of the [num_tokens * H, 576] query matrix and a chunk's tokens follow each
// other, so 128 consecutive rows of that matrix are one tensor-core tile whatever H is: with 16 heads a tile holds
// eight tokens of the request, which share every key.  The causal mask is the only thing that differs between the tokens
// of a tile.  (Sparse attention: one query per tile, its keys are its own.)
//
// The pair.  O of 128 rows x 512 values in f32 fills tensor memory, so the values are split over two CTAs; if each
// computed S = Q K^T for itself, 576 of 1088 multiplications would be done twice (measured, single calls after a pause:
// 1.48 ms for 512 tokens x 64 heads at 16k context, against 1.15 ms for the first form of this kernel and 1.10 ms now).  Here the two are a cluster: of every 128 keys (a step) each computes S and
// P for its own 64-key page, and copies P to the other through distributed shared memory (16 KB a step); both multiply
// the whole P (128 rows x 128 keys) with their half of the values.  Softmax bases have to agree: the rows' maxima of the
// two pages are exchanged first (one f32 a row).
//
// Per step and CTA: Q K^T of 64 keys (36 products of N = 64, ~1340 cycles), P V of 128 keys (8 of N = 256, 1024), into
// shared memory the own page's nine 64-dim column blocks (72 KB) and this half's four of the other page (32 KB).
// What bounds it: over bf16 rows (~4000 cycles a step) the shared-memory port, busy for ~2800 of them with the copies in,
// the products' operands and P, and the exchange between the CTAs; over quantised rows (~6000) the warps that turn codes
// into bf16.  And the instruction cache: the roles' loops together have to fit it, so most are kept rolled up.
// Measured, calls back to back: 512 tokens x 64 heads at 16k context 1.22 ms (972 TFLOP/s), a prompt of 2048 tokens x 128
// heads 0.72 ms (806); both run against the power limit then (single calls after a pause took 1.10 and 0.65 ms).  64 queries
// x 128 heads over 2048 selected quantised rows each 74 us (491), 1024 queries x 64 heads 0.80 ms (366: 64 heads fill half a
// tile).
//
// Tensor memory: O_v [0, 256), S [256, 320), six of Q's nine column blocks [320, 512).  Shared memory: the other
// three (48 KB), P of both pages (32 KB), blocks X (16 KB) and Y (24 KB) of the own page, needed until Q K^T is past
// them, and V stages (32 KB: four value blocks of a page) until its P V is done: two for the own page, which Q K^T
// reads a step before P V does, one for the other page.  Blocks are 64 rows x 64 dims, 128B-swizzled: the same bytes
// are the K-major B of Q K^T and the MN-major B of P V.
//
// Quantised rows become bf16 on their way in: eight warps load a row's codes with 16-byte loads, turn them into bf16
// (exact: a code has four significant bits and its scale is a power of two) and store them in the swizzled layout; the
// other page's half is converted again rather than copied (its place is free only when X and Y are wanted for the next
// step).  bf16 rows come by TMA: whole 64-token pages as 64-row boxes, a page's visible part by gather4.
//
// Roles (16 warps): 0-7 fill the blocks and move Q into tensor memory; 8-11 softmax and epilogue, one row per thread;
// 12 issues the products (the whole warp, so that the compiler keeps the issue uniform: with elect.sync one product of
// N = 64 goes out every ~32 cycles, against ~60 from a thread chosen by its index); 13 hands out units and looks pages
// up, steps ahead.  Order of products: Q K^T of step g, then P V of step g - 1, so that the tensor core has P V to do
// while the softmax reads S.  All waits are bounded; bad rows set the device error word and are skipped.
#include "mla_packed.cuh"

namespace dsa {
namespace {

using namespace packed;

constexpr int kIssueWarp = kFillWarps + 4, kLookupWarp = kIssueWarp + 1;
constexpr int kThreads = 32 * 16;
// Registers a thread by warpgroup, 4 x 128 in all.  Spilled ones cost more than elsewhere: they miss the small L1
// left beside 220 KB of shared memory (300 bytes of spill loads in the quantised fill cost a prefill of 1024 queries a
// tenth).
template <Source kSrc>
struct Regs {
  static constexpr bool kQuant = kSrc != kPagesBf16;
  static constexpr int kFill = kQuant ? 136 : 96, kSoftmax = kQuant ? 128 : 184, kIssue = kQuant ? 112 : 136;
};

template <int kRegs>
__device__ __forceinline__ void set_registers() {  // of this warp's warpgroup; 128 at launch
  if constexpr (kRegs > 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  if constexpr (kRegs < 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// ---- cluster
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_address(const void* mine, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(mine)), "r"(rank));
  return a;
}
// stores into the other CTA whose bytes are counted on its barrier `bar` once they are there
__device__ __forceinline__ void st_async4(uint32_t dst, uint32_t v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(dst), "r"(v), "r"(bar) : "memory");
}
// `bytes` of this CTA's shared memory into the other's, counted likewise
__device__ __forceinline__ void copy_to_peer(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}
// Warp-collective bounded wait, as warp_wait, for a phase that the other CTA takes part in: it acquires at
// cluster scope (a fence after a plain wait costs several hundred cycles more).
__device__ __forceinline__ bool cluster_wait(uint64_t* bar, uint32_t parity, int* err, volatile int* abort_flag) {
  const uint32_t b = smem_u32(bar);
  bool ok = false;
  long long t0 = 0;
  for (uint32_t n = 0; !ok; ++n) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(b), "r"(parity)
        : "memory");
    ok = done != 0;
    if (ok) break;
    if (n == 0) t0 = clock64();
    if (*abort_flag) break;
    if (clock64() - t0 > kWaitCycles) {
      raise_error(err, DSA_DEVERR_TIMEOUT);
      *abort_flag = 1;
      break;
    }
  }
  return __all_sync(0xFFFFFFFFu, ok);
}
__device__ __forceinline__ void umma_ss_acc(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)acc));
}
// arrive on `bar` of both CTAs once every product issued so far by this thread has completed
__device__ __forceinline__ void mma_commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

template <Source kSrc>
__global__ void __launch_bounds__(kThreads, 1)
    mla_pair_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap rmap,
                    const __grid_constant__ CUtensorMap pmap, const Params p) {
  constexpr bool kQuant = kSrc != kPagesBf16;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t v = cluster_rank();  // this CTA's value half, and its page of each step
  uint8_t* q_s = smem + OFF_Q;
  uint8_t* x_st = smem + OFF_X;
  uint8_t* y_st = smem + OFF_Y;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* xy_full = bars + 0;     // [2] X and Y of the own page in place, masks published
  uint64_t* vo_full = bars + 2;     // [2] V of the own page
  uint64_t* vp_full = bars + 4;     // [2] V of the other page
  uint64_t* land = bars + 6;        // [2] rows landed, to be looked over before the above: own page
  uint64_t* land_p = bars + 8;      // [2] other page
  uint64_t* x_empty = bars + 10;    // Q K^T is past the X blocks
  uint64_t* y_empty = bars + 11;    // ... past the Y blocks
  uint64_t* vo_empty = bars + 12;   // [2] P V of the own page done
  uint64_t* vp_empty = bars + 14;   // P V of the other page done
  uint64_t* q_stage = bars + 15;
  uint64_t* q_read = bars + 16;
  uint64_t* q_full = bars + 17;
  uint64_t* q_empty = bars + 18;
  uint64_t* s_full = bars + 19;
  uint64_t* s_empty = bars + 20;
  uint64_t* p_full = bars + 21;     // P of both pages written (the other CTA's counted in bytes)
  uint64_t* pv_done = bars + 22;    // P V of the step done, in both CTAs
  uint64_t* fin = bars + 23;
  uint64_t* ep_last = bars + 24;
  uint64_t* r_full = bars + 25;     // [kSlots]
  uint64_t* r_empty = bars + 29;    // [kSlots]
  uint64_t* u_full = bars + 33;     // [kUnitSlots]
  uint64_t* u_empty = bars + 35;    // [kUnitSlots]
  uint64_t* x_bar = bars + 37;      // [4] the other CTA's values of 32 rows have come
  uint64_t* mail = bars + 41;       // [4] a unit from CTA 0 has come
  uint8_t* masks = smem + OFF_MASK;
  uint8_t* poisons = smem + OFF_POISON;
  float* stats = reinterpret_cast<float*>(smem + OFF_STATS);
  volatile float* peer_max = reinterpret_cast<volatile float*>(smem + OFF_MAX);
  Unit* unit_ring = reinterpret_cast<Unit*>(smem + OFF_UNIT);
  int32_t* row_ring = reinterpret_cast<int32_t*>(smem + OFF_ROWS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 8);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = p.tiles * p.nsplit, clusters = gridDim.x / 2;
  griddep_launch_dependents();

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&xy_full[i], kFillWarps);
      mbar_init(&vo_full[i], kFillWarps);
      mbar_init(&vp_full[i], kFillWarps);
      mbar_init(&land[i], kFillWarps);
      mbar_init(&land_p[i], kFillWarps);
    }
    mbar_init(x_empty, 1);
    mbar_init(y_empty, 1);
    mbar_init(&vo_empty[0], 1);
    mbar_init(&vo_empty[1], 1);
    mbar_init(vp_empty, 1);
    mbar_init(q_stage, 1);
    mbar_init(q_read, kFillWarps);
    mbar_init(q_full, kFillWarps);
    mbar_init(q_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(s_empty, 4);
    mbar_init(p_full, 4);
    mbar_init(pv_done, 2);
    mbar_init(fin, 1);
    mbar_init(ep_last, 4);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&r_full[i], 1);
      mbar_init(&r_empty[i], kFillWarps);
      mbar_init(&x_bar[i], 1);
      mbar_init(&mail[i], 1);
    }
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_empty[i], kIssueWarp + 1);  // fill, softmax, issue
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();

  auto take_unit = [&](int k, Unit& x) -> bool {
    if (!warp_wait(&u_full[k % kUnitSlots], (k / kUnitSlots) & 1, p.err, abort_flag)) return false;
    x = unit_ring[k % kUnitSlots];
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_empty[k % kUnitSlots]);
    return x.rows > 0;
  };
  auto last_unit = [&](int k, bool& last) -> bool {
    if (!warp_wait(&u_full[(k + 1) % kUnitSlots], ((k + 1) / kUnitSlots) & 1, p.err, abort_flag)) return false;
    last = unit_ring[(k + 1) % kUnitSlots].rows < 0;
    return true;
  };
  auto v_own = [&](int g) { return smem + OFF_V + (g & 1) * V_BYTES; };
  uint8_t* v_peer = smem + OFF_V + 2 * V_BYTES;

  if (warp < kFillWarps) {
    set_registers<Regs<kSrc>::kFill>();
    // ------------------------------------------------------------------ copies, and Q into tensor memory
    const int quarter = warp & 3, part = warp >> 2;
    const uint32_t my_lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const int key = warp * kKeysPerWarp + (lane & 7);
    int gi = 0, ui = 0;  // steps and units of this CTA
    uint32_t nland[2] = {0u, 0u}, nland_p[2] = {0u, 0u};
    bool ok = true, staged = false;
    Unit x;
    for (; ok && take_unit(ui, x);) {
      const int nsteps = (x.hi - x.lo + 2 * kTile - 1) / (2 * kTile);

      // --- Quantised rows.  A warp has eight keys of either page, pair q its keys 2 q + half; a lane has 16 codes of a
      // row in one half of the values.  Lane l has the scale of key l / 4, group l % 4.  Codes are fetched into L2 some
      // conversions ahead of their load, unless they are there (the launch decides; loaded a group ahead into the registers that
      // the last group leaves, decode of 64 queries takes 79 us for 73).  A key without a row reads row 0.
      const int half = (lane >> 2) & 1, l16 = (lane & 3) | (lane >> 3) << 2;  // eight lanes: four pieces of both rows of a pair
      uint4 code[4];
      float sc_own = 1.0f;
      uint32_t seen_own = 0u, bad_own = 0u;  // lanes: key with a row; no row, or a scale that is no power of two
      auto row_at = [&](int g, int which, int k8) -> int { return row_ring[(g % kSlots * 2 + which) * kTile + warp * kKeysPerWarp + k8]; };
      auto load_codes = [&](int g, int which, uint32_t h) {
        const uint8_t* base = p.data + 256 * h + 16 * l16;
#pragma unroll
        for (int q = 0; q < 4; ++q) code[q] = load16_here(base + (int64_t)max(0, row_at(g, which, 2 * q + half)) * kLatentBytes);
      };
      auto fetch = [&](int g, int which, uint32_t h) {
        if (kSrc == kSelected && !p.cold) return;
        const uint8_t* a = p.data + (int64_t)max(0, row_at(g, which, lane >> 2)) * kLatentBytes + 256 * h + 64 * (lane & 3);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a));  // (a row's 256 bytes: four lanes)
      };
      auto load_scales = [&](int g, int which) -> float {
        return loadf_here(p.scale + (int64_t)max(0, row_at(g, which, lane >> 2)) * 4 + (lane & 3));
      };
      auto check_own = [&](int g) {
        const bool none = row_at(g, 0, lane >> 2) < 0;
        bad_own = __ballot_sync(0xFFFFFFFFu, none || !latent_scale_ok(sc_own));
        seen_own = ~__ballot_sync(0xFFFFFFFFu, none);
      };
      // The 16 codes of each pair's row in `code`, of value half h, into the row's blocks: `dst` is the lane's 64-dim block, pieces
      // 2 (l16 % 4) and the next; the two rows of a pair differ in bit 0, so eight lanes store to all eight bank groups.
      // partly: only some of the tile's tokens see the rows, and a NaN must not reach the others through 0 * NaN in
      // P V: it becomes zero and its row is noted, so that the softmax makes the weights of those that see it NaN
      // (elsewhere a NaN takes its natural course).
      auto put_all = [&](float sc, uint32_t bad, uint32_t h, bool partly, uint8_t* dst, uint32_t& nan_rows) {
        auto put = [&](auto plain, int q) {
          constexpr bool kPlain = decltype(plain)::value;
          const int k8 = 2 * q + half, r = warp * kKeysPerWarp + k8;
          uint32_t w[4] = {code[q].x, code[q].y, code[q].z, code[q].w};
          float my_sc = __shfl_sync(0xFFFFFFFFu, sc, k8 * 4 + 2 * (int)h + (l16 >> 3));
          if (!kPlain && ((bad >> (4 * k8)) & 0xFu)) {
            w[0] = w[1] = w[2] = w[3] = 0u;
            my_sc = 1.0f;
          }
          uint32_t b[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) decode4(w[i], make_float2(my_sc, my_sc), b[2 * i], b[2 * i + 1]);
          if (!kPlain && partly) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if ((b[i] & 0x7F80u) == 0x7F80u) { b[i] &= 0xFFFF0000u; nan_rows |= 1u << k8; }
              if ((b[i] & 0x7F800000u) == 0x7F800000u) { b[i] &= 0xFFFFu; nan_rows |= 1u << k8; }
            }
          }
          const uint32_t piece = (uint32_t)(l16 & 3) * 2u, x7 = (uint32_t)(r & 7);
          *reinterpret_cast<uint4*>(dst + r * 128 + ((piece ^ x7) << 4)) = make_uint4(b[0], b[1], b[2], b[3]);
          *reinterpret_cast<uint4*>(dst + r * 128 + (((piece + 1u) ^ x7) << 4)) = make_uint4(b[4], b[5], b[6], b[7]);
        };
        if (bad == 0u && !partly) {
#pragma unroll
          for (int q = 0; q < 4; ++q) put(Flag<true>(), q);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) put(Flag<false>(), q);
        }
      };
      if (kQuant && nsteps > 0) {
        if (!(ok = warp_wait(&r_full[gi % kSlots], (gi / kSlots) & 1, p.err, abort_flag))) break;
        sc_own = load_scales(gi, 0);
        fetch(gi, 0, v);
        check_own(gi);
      }

      // --- Q of the unit: places 0 .. 2 of the block order to shared memory, the other six through X, the
      // first two thirds of Y and the own page's two V stages to tensor memory
      auto stage_at = [&](int b) { return b == 0 ? x_st : b == 1 ? y_st : smem + OFF_V + (b - 2) * Q_CHUNK; };
      auto vo_free = [&](int g) { return g < 2 || warp_wait(&vo_empty[g & 1], ((g / 2) - 1) & 1, p.err, abort_flag); };
      if (ui >= 1 && !(ok = warp_wait(q_empty, (ui - 1) & 1, p.err, abort_flag))) break;
      if (!(ok = vo_free(gi)) || !(ok = vo_free(gi + 1))) break;
      if (tid == 0) {
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(q_stage, kChunks * Q_CHUNK);
#pragma unroll
        for (int c = kSmemQ; c < kChunks; ++c) tma_load_2d(stage_at(c - kSmemQ), &qmap, q_stage, block_of(c, v) * 64, x.row0);
        for (int c = 0; c < kSmemQ; ++c) tma_load_2d(q_s + c * Q_CHUNK, &qmap, q_stage, block_of(c, v) * 64, x.row0);
        staged = true;
      }
      tc_fence_after();
      if (!(ok = warp_wait(q_stage, ui & 1, p.err, abort_flag))) break;
      staged = false;
      {
        const int r = quarter * 32 + lane;
        // (written out it makes the quantised forms spill: sparse prefill of 1024 queries 825 -> 833 us; rolled up it costs
        // the bf16 form more than it saves: 512 tokens at 16k context 1101 -> 1116 us)
#pragma unroll(kQuant ? 1 : 6)
        for (int b = 0; b < 6; ++b) {  // this warp's half (64 bytes) of the row's block
          const uint8_t* src = stage_at(b) + r * 128;
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 y = *reinterpret_cast<const uint4*>(src + (((part * 4 + e) ^ (r & 7)) << 4));
            w[4 * e] = y.x; w[4 * e + 1] = y.y; w[4 * e + 2] = y.z; w[4 * e + 3] = y.w;
          }
          tmem_st16(my_lanes + TM_Q + b * 32 + part * 16, w);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(q_full);
        mbar_arrive(q_read);
      }
      if (!(ok = warp_wait(q_read, ui & 1, p.err, abort_flag))) break;
      ++ui;

      if constexpr (kQuant) {
        // Three groups of codes a step, by one piece of code (three copies of it do not fit the instruction cache beside the
        // other roles' loops: prefill of 1024 queries 871 -> 1040 us): the own page's other half into X1 and Y, its this
        // half into V, and, a step behind, the other page's this half into its V.
#pragma unroll 1
        for (int j = 0; j <= nsteps && ok; ++j) {
          const int s = gi & 1, slot = gi % kSlots;
          float sc_next = 1.0f;
          uint32_t nan_rows = 0u;
#pragma unroll 1
          for (int part3 = j < nsteps ? 0 : 2; part3 < (j > 0 ? 3 : 2); ++part3) {
            const bool other = part3 == 2;
            const int g = other ? gi - 1 : gi;                       // step of the rows
            const uint32_t h = part3 == 0 ? v ^ 1u : v;              // their half
            const int base = x.lo + (2 * (other ? j - 1 : j) + (other ? 1 - (int)v : (int)v)) * kTile;
            const bool partly = kSrc != kSelected && base + kTile - 1 > x.tok0 && x.hi - 1 > max(x.tok0, base - 1);
            float sc = sc_own;
            uint32_t bad = bad_own;
            if (other) {
              sc = load_scales(g, 1);
              bad = __ballot_sync(0xFFFFFFFFu, row_at(g, 1, lane >> 2) < 0);  // no row; below: or a bad scale
            }
            load_codes(g, other, h);
            uint8_t* dst = v_peer;
            if (part3 == 0) {
              if (gi >= 1 && (!(ok = warp_wait(x_empty, (gi - 1) & 1, p.err, abort_flag)) || !(ok = warp_wait(y_empty, (gi - 1) & 1, p.err, abort_flag)))) break;
              // X0: the RoPE part as it is, in the background
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int r8 = 4 * i + (lane >> 3);
                const int r = warp * kKeysPerWarp + r8;
                cp_async_16(smem_u32(x_st + r * 128 + (((lane & 7) ^ (r & 7)) << 4)),
                            p.data + (int64_t)max(0, row_at(gi, 0, r8)) * kLatentBytes + kDv + 16 * (lane & 7),
                            ((bad >> (4 * r8)) & 0xFu) ? 0u : 16u);
              }
              dst = (l16 >> 2) == 3 ? x_st + K_CHUNK - 3 * K_CHUNK : y_st;
            } else if (part3 == 1) {
              if (!(ok = vo_free(gi))) break;
              dst = v_own(gi);
            } else {
              if (g >= 1 && !(ok = warp_wait(vp_empty, (g - 1) & 1, p.err, abort_flag))) break;
              // (of either half: the whole row is skipped, and a NaN code left of it would reach O as 0 * NaN)
              bad |= __ballot_sync(0xFFFFFFFFu, !latent_scale_ok(sc));
            }
            put_all(sc, bad, h, partly, dst + (l16 >> 2) * K_CHUNK, nan_rows);
            if (part3 == 0) continue;
            if (part3 == 1) {
              if (j + 1 < nsteps) {
                if (!(ok = warp_wait(&r_full[(gi + 1) % kSlots], ((gi + 1) / kSlots) & 1, p.err, abort_flag))) break;
                sc_next = load_scales(gi + 1, 0);
                fetch(gi + 1, 0, v ^ 1u);
                fetch(gi + 1, 0, v);
              }
              fetch(gi, 1, v);
              const uint32_t poison = __reduce_or_sync(0xFFFFFFFFu, nan_rows);
              if (lane == 0) {
                uint32_t valid = 0xFFu;
                if (bad) {
                  bool flag = false;
                  for (int r8 = 0; r8 < kKeysPerWarp; ++r8)
                    if ((bad >> (4 * r8)) & 0xFu) {
                      valid &= ~(1u << r8);
                      flag |= (seen_own >> (4 * r8)) & 1u;
                    }
                  if (flag) raise_error(p.err, DSA_DEVERR_SCALE);
                }
                masks[slot * 8 + warp] = (uint8_t)valid;
                poisons[slot * 8 + warp] = (uint8_t)(poison & valid);
              }
              cp_async_wait_all();
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (part3 == 1) {
                mbar_arrive(&xy_full[s]);
                mbar_arrive(&vo_full[s]);
              } else {
                mbar_arrive(&vp_full[g & 1]);
                mbar_arrive(&r_empty[g % kSlots]);
              }
            }
          }
          if (!ok) break;
          if (j + 1 < nsteps) {
            sc_own = sc_next;
            check_own(gi + 1);
          }
          if (j < nsteps) ++gi;
        }
      } else {
      // --- copies.  A page: its first position, its number (-1: none), its rows that may be read.
      struct Page {
        int base, page;
        uint32_t may[2];
      };
      auto page_of = [&](int g, int j, int which) -> Page {  // which: 0 own, 1 the other
        const int32_t* e = row_ring + g % kSlots * 8;
        return Page{x.lo + (2 * j + (which ? 1 - (int)v : (int)v)) * kTile, e[which], {(uint32_t)e[2 + 2 * which], (uint32_t)e[3 + 2 * which]}};
      };
      auto row_of = [&](const Page& a) -> int {
        const bool may = (a.may[key >> 5] >> (key & 31)) & 1u;
        return a.page >= 0 && may && a.base + key < x.hi ? a.page * kTile + key : -1;
      };
      auto is_whole = [&](const Page& a) { return a.page >= 0 && (a.may[0] & a.may[1]) == ~0u && a.base + kTile <= x.hi; };
      // rows that only some of the tile's tokens see: a NaN there must not reach the others through 0 * NaN in P V
      auto is_partly = [&](const Page& a) { return a.base + kTile - 1 > x.tok0 && x.hi - 1 > max(x.tok0, a.base - 1); };
      auto arm = [&](uint64_t* bar, bool whole, int blocks) {
        if (lane != 0) return;
        if (!whole)
          mbar_arrive_expect_tx(bar, kKeysPerWarp * 128 * blocks);
        else if (warp == 0)
          mbar_arrive_expect_tx(bar, K_CHUNK * blocks);
        else
          mbar_arrive(bar);
      };
      // places lo .. hi - 1 of the block order
      auto copy = [&](const Page& a, bool whole, int row, int lo, int hi, uint8_t* dst, uint64_t* bar) {
        if (whole) {
          if (warp == 0 && lane == 0)
#pragma unroll 1
            for (int c = lo; c < hi; ++c) tma_load_2d(dst + (c - lo) * K_CHUNK, &pmap, bar, block_of(c, v) * 64, a.page * kTile);
          return;
        }
#pragma unroll 1
        for (int g4 = 0; g4 < 2; ++g4) {
          const int rc = row >= 0 ? row : p.oob_row;
          const int r0 = __shfl_sync(0xFFFFFFFFu, rc, 4 * g4), r1 = __shfl_sync(0xFFFFFFFFu, rc, 4 * g4 + 1);
          const int r2 = __shfl_sync(0xFFFFFFFFu, rc, 4 * g4 + 2), r3 = __shfl_sync(0xFFFFFFFFu, rc, 4 * g4 + 3);
          if (lane == 0)
#pragma unroll 1
            for (int c = lo; c < hi; ++c)
              tma_gather4(dst + (c - lo) * K_CHUNK + (warp * kKeysPerWarp + 4 * g4) * 128, &rmap, bar, block_of(c, v) * 64, r0, r1, r2, r3);
        }
      };
      // Looks over one 64-dim block's 128 bytes of eight rows (four lanes a row): whether values are not finite; `zero`
      // makes those zero.  Returns a bit per row of this warp.
      auto scan = [&](const Page& a, uint8_t* block, bool zero) -> uint32_t {
        const int r = warp * kKeysPerWarp + (lane >> 2);
        bool f = false;
        if (a.base + r > x.tok0 && a.base + r < x.hi) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint4* at = reinterpret_cast<uint4*>(block + r * 128 + (((lane & 3) * 2 + e) << 4));
            const uint4 y = *at;
            uint32_t w[4] = {y.x, y.y, y.z, y.w};
            bool g = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if ((w[k] & 0x7F80u) == 0x7F80u) { w[k] &= 0xFFFF0000u; g = true; }
              if ((w[k] & 0x7F800000u) == 0x7F800000u) { w[k] &= 0xFFFFu; g = true; }
            }
            if (g && zero) *at = make_uint4(w[0], w[1], w[2], w[3]);
            f |= g;
          }
        }
        const uint32_t b = __ballot_sync(0xFFFFFFFFu, f);
        uint32_t rows = 0u;
#pragma unroll
        for (int k = 0; k < kKeysPerWarp; ++k) rows |= (b >> (4 * k)) & 0xFu ? 1u << k : 0u;
        return rows;
      };
      // the other page's V of step j (CTA step g)
      Page peer = {0, -1, {0u, 0u}};
      auto copy_peer = [&](int g) -> bool {
        const int s = g & 1;
        const bool whole = is_whole(peer), partly = is_partly(peer);
        if (g >= 1 && !warp_wait(vp_empty, (g - 1) & 1, p.err, abort_flag)) return false;
        uint64_t* bar = partly ? &land_p[s] : &vp_full[s];
        if (lane == 0) fence_proxy_async_smem();
        arm(bar, whole, kVBlocks);
        __syncwarp();
        copy(peer, whole, row_of(peer), 5, 9, v_peer, bar);
        if (partly) {
          if (!warp_wait(&land_p[s], nland_p[s] & 1, p.err, abort_flag)) return false;
          ++nland_p[s];
#pragma unroll 1
          for (int c = 0; c < kVBlocks; ++c) scan(peer, v_peer + c * K_CHUNK, true);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&vp_full[s]);
        }
        return true;
      };

      // Order by when the places become free: X and Y of step g while Q K^T of g - 1 runs, then, as P V of g - 2 goes
      // on, V of the own page of g and of the other page of g - 1.
      for (int j = 0; j < nsteps; ++j, ++gi) {
        const int s = gi & 1, slot = gi % kSlots;
        if (!(ok = warp_wait(&r_full[slot], (gi / kSlots) & 1, p.err, abort_flag))) break;
        const Page own = page_of(gi, j, 0), next_peer = page_of(gi, j, 1);
        const int row = row_of(own);
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, row >= 0) & 0xFFu;
        if (lane == 0) mbar_arrive(&r_empty[slot]);
        const bool whole = is_whole(own), partly = is_partly(own);
        uint64_t* xy_bar = partly ? &land[s] : &xy_full[s];
        uint64_t* vo_bar = partly ? &land[s] : &vo_full[s];
        if (gi >= 1 && !(ok = warp_wait(x_empty, (gi - 1) & 1, p.err, abort_flag))) break;
        if (lane == 0) {
          masks[slot * 8 + warp] = (uint8_t)valid;
          if (!partly) poisons[slot * 8 + warp] = 0;
          fence_proxy_async_smem();
        }
        arm(xy_bar, whole, partly ? kChunks : kXBlocks + kYBlocks);
        __syncwarp();
        copy(own, whole, row, 0, 2, x_st, xy_bar);
        if (gi >= 1 && !(ok = warp_wait(y_empty, (gi - 1) & 1, p.err, abort_flag))) break;
        copy(own, whole, row, 2, 5, y_st, xy_bar);
        if (!(ok = vo_free(gi))) break;
        if (!partly) arm(vo_bar, whole, kVBlocks);
        __syncwarp();
        copy(own, whole, row, 5, 9, v_own(gi), vo_bar);
        if (partly) {
          if (!(ok = warp_wait(&land[s], nland[s] & 1, p.err, abort_flag))) break;
          ++nland[s];
          // values that are not finite become zero in the V blocks and their row is noted: the softmax makes
          // the weights of the tokens that see it NaN.  (In X and Y a NaN only reaches logits, of hidden keys masked ones.)
          uint32_t poison = 0u;
#pragma unroll 1
          for (int c = 1; c < kChunks; ++c)
            poison |= scan(own, (c == 1 ? x_st : c < 5 ? y_st - 2 * K_CHUNK : v_own(gi) - 5 * K_CHUNK) + c * K_CHUNK, c >= 5);
          if (lane == 0) poisons[slot * 8 + warp] = (uint8_t)poison;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&xy_full[s]);
            mbar_arrive(&vo_full[s]);
          }
        }
        if (j > 0 && !(ok = copy_peer(gi - 1))) break;
        peer = next_peer;
      }
      if (ok) ok = copy_peer(gi - 1);
      }
      bool last;
      if (!ok || !(ok = last_unit(ui - 1, last))) break;
      if (last) {
        if (!(ok = warp_wait(ep_last, 0, p.err, abort_flag))) break;
        tc_fence_after();
        store_o(p, x, my_lanes, quarter, 64 + 96 * part, 160 + 96 * part, smem + OFF_V + warp * kStageBytes, stats[quarter * 32 + lane], nsteps > 0);
        tc_fence_before();
      }
    }
    // gave up: copies in flight must land before the CTA exits
    if (!ok && staged) mbar_wait(q_stage, ui & 1, p.err, nullptr);
    if (!ok && !kQuant && lane == 0) {
      for (int t = gi > 0 ? gi - 1 : 0; t <= gi; ++t) {
        mbar_wait(&xy_full[t & 1], (uint32_t)((t / 2) & 1), p.err, nullptr, kWaitCycles / 16);
        mbar_wait(&vo_full[t & 1], (uint32_t)((t / 2) & 1), p.err, nullptr, kWaitCycles / 16);
        mbar_wait(&vp_full[t & 1], (uint32_t)((t / 2) & 1), p.err, nullptr, kWaitCycles / 16);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_wait(&land[i], nland[i] & 1, p.err, nullptr, kWaitCycles / 16);
        mbar_wait(&land_p[i], nland_p[i] & 1, p.err, nullptr, kWaitCycles / 16);
      }
    }
  } else if (warp < kIssueWarp) {
    set_registers<Regs<kSrc>::kSoftmax>();
    // ------------------------------------------------------------------ softmax and epilogue
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t peer_x_bar = peer_address(&x_bar[quarter], v ^ 1u), peer_p_full = peer_address(p_full, v ^ 1u);
    uint8_t* p_mine = smem + p_offset((int)v, quarter);  // P of this warp's rows
    uint8_t* p_row = p_mine + (lane >> 3) * 1024 + (lane & 7) * 16;
    const uint32_t peer_p = peer_address(p_mine, v ^ 1u);
    const uint32_t peer_slot = peer_address(smem + OFF_MAX + r * 4, v ^ 1u);
    int gi = 0, nx = 0;
    bool ok = true;
    // The other CTA's value of this row.  The barrier is armed before the own value goes out: the other CTA, which waits
    // for it, cannot be a round ahead.
    auto exchange = [&](float mine, float& other) -> bool {
      if (lane == 0) mbar_arrive_expect_tx(&x_bar[quarter], 128);
      __syncwarp();
      const int buf = (nx & 1) * kRows;
      st_async4(peer_slot + buf * 4, __float_as_uint(mine), peer_x_bar);
      if (!cluster_wait(&x_bar[quarter], nx & 1, p.err, abort_flag)) return false;
      ++nx;
      other = peer_max[buf + r];
      return true;
    };
    Unit x;
    for (int ui = 0; ok && take_unit(ui, x); ++ui) {
      const int nsteps = (x.hi - x.lo + 2 * kTile - 1) / (2 * kTile);
      // last position this row sees (kSelected: the keys' own mask tells)
      const int limit = r >= x.rows ? -1 : kSrc == kSelected ? 0x7FFFFFFF : x.tok0 + (x.h0 + r) / p.H;
      float m_used = -INFINITY, l = 0.0f;
      for (int j = 0; j < nsteps; ++j, ++gi) {
        const int slot = gi % kSlots;
        if (!(ok = warp_wait(s_full, gi & 1, p.err, abort_flag))) break;
        if (!(ok = warp_wait(&xy_full[gi & 1], (gi / 2) & 1, p.err, abort_flag))) break;  // (long past: orders the masks)
        tc_fence_after();
        uint32_t sv[64];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld16(lane_base + TM_S + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&sv[16 * c]));
        uint64_t valid = *reinterpret_cast<const volatile uint64_t*>(masks + slot * 8);
        const uint64_t poison = *reinterpret_cast<const volatile uint64_t*>(poisons + slot * 8);
        const int d = limit - (x.lo + (2 * j + (int)v) * kTile);  // this row sees the page's keys 0 .. d
        if (d < 63) valid &= d < 0 ? 0ull : (2ull << d) - 1ull;
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty);
        if (!__all_sync(0xFFFFFFFFu, valid == ~0ull && poison == 0ull)) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!((valid >> c) & 1u)) sv[c] = 0xFF800000u;
          if (valid & poison) sv[0] = 0x7FC00000u;  // (one NaN weight makes the row's results NaN)
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(sv[c]);
#pragma unroll
        for (int c = 4; c < 64; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(sv[c]));
        float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        float other;
        if (!(ok = exchange(mt, other))) break;
        mt = fmaxf(mt, other);
        // Lazy rescale: a row's base m_used moves only when its maximum exceeds it by more than 2^8 (P stays
        // <= 256); the warp takes the step together, since the tensor-memory accesses are warp-collective.
        const bool rescale = __any_sync(0xFFFFFFFFu, mt > m_used + 8.0f);
        float f = 1.0f;
        if (rescale) {
          const float m_new = mt > m_used + 8.0f ? mt : m_used;  // (a row's base depends on that row alone)
          f = m_new == -INFINITY ? 1.0f : exp2f(m_used - m_new);  // 0 when m_used = -inf
          l *= f;
          m_used = m_new;
        }
        uint32_t pk[32];
        const float nsub = m_used == -INFINITY ? 0.0f : -m_used;
        float2 ps[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), ns2 = make_float2(nsub, nsub);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 e = fma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sc2, ns2);
          const float2 w = make_float2(fast_exp2(e.x), fast_exp2(e.y));
          // P is rounded to bf16 (2^-8 of each weight): both operands of a product have one type, and V is bf16.  The
          // normaliser sums the weights before that.
          ps[(c >> 1) & 1] = add2(ps[(c >> 1) & 1], w);
          const __nv_bfloat162 b = __floats2bfloat162_rn(w.x, w.y);
          pk[c >> 1] = *reinterpret_cast<const uint32_t*>(&b);
        }
        const float2 pt = add2(ps[0], ps[1]);
        l += pt.x + pt.y;
        // O and both CTAs' P buffers are free once the previous step's P V has completed in both
        if (gi >= 1 && !(ok = cluster_wait(pv_done, (gi - 1) & 1, p.err, abort_flag))) break;
#pragma unroll
        for (int kc = 0; kc < 8; ++kc)
          *reinterpret_cast<uint4*>(p_row + kc * 128) = make_uint4(pk[4 * kc], pk[4 * kc + 1], pk[4 * kc + 2], pk[4 * kc + 3]);
        // to the other CTA as one 4 KB copy (stores of 16 bytes got through at ~9 bytes a cycle)
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) copy_to_peer(peer_p, p_mine, (uint32_t)kWarpPBytes, peer_p_full);
        if (rescale && j > 0) {
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < kHalf; c0 += 32) {
            uint32_t o[32];
            tmem_ld16(lane_base + TM_O + c0, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
            tmem_ld16(lane_base + TM_O + c0 + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tmem_st16(lane_base + TM_O + c0, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
            tmem_st16(lane_base + TM_O + c0 + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(p_full, (uint32_t)kWarpPBytes);  // and the other CTA's P of these 32 rows
      }
      if (!ok) break;
      float other;
      if (!(ok = exchange(l, other))) break;
      l = v ? other + l : l + other;
      if (nsteps > 0 && !(ok = cluster_wait(pv_done, (gi - 1) & 1, p.err, abort_flag))) break;
      tc_fence_after();
      // a row that saw nothing: 0 and -inf; NaN stays NaN
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const float lse = l == 0.0f ? -INFINITY : (m_used + log2f(l)) * 0.69314718055994531f;
      bool last;
      if (!(ok = last_unit(ui, last))) break;
      if (last) {
        stats[r] = inv;
        __syncwarp();
        if (lane == 0) mbar_arrive(ep_last);
      }
      store_o(p, x, lane_base, quarter, 0, last ? 64 : kHalf, smem + stage_offset((int)v, quarter), inv, nsteps > 0);
      if (v == 0 && r < x.rows) {
        if (x.splits == 1) {
          if (p.lse) p.lse[(int64_t)x.row0 + r] = lse;
        } else {
          p.part_lse[(int64_t)x.prow + r] = lse;
        }
      }
      tc_fence_before();
    }
  } else {
    set_registers<Regs<kSrc>::kIssue>();
    if (warp == kIssueWarp) {
      // ------------------------------------------------------------------ the products
      const uint32_t idesc_s = idesc_f16(1u, 0u, (uint32_t)kRows, (uint32_t)kTile);
      const uint32_t idesc_o = idesc_f16(1u, 1u, (uint32_t)kRows, (uint32_t)kHalf);
      const uint64_t qd = sw128_desc(smem_u32(q_s), 16, 1024);
      const uint64_t xd = sw128_desc(smem_u32(x_st), 16, 1024), yd = sw128_desc(smem_u32(y_st), 16, 1024);
      const uint32_t d_s = tmem + TM_S, a_q = tmem + TM_Q, d_o = tmem + TM_O;
      int gi = 0, ui = 0;
      bool ok = true;
      // P V of CTA step g: the own page, then the other
      auto issue_pv = [&](int g, bool first) -> bool {
        if (!cluster_wait(p_full, g & 1, p.err, abort_flag)) return false;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t pd = noswz_desc(smem_u32(smem + OFF_P + v * P_BYTES), 128, 1024);
        const uint64_t vd = sw128_desc(smem_u32(v_own(g)), K_CHUNK, 1024);
        if (elect_one()) {
          if (first)
            umma_ss<0>(d_o, pd, vd, idesc_o);
          else
            umma_ss<1>(d_o, pd, vd, idesc_o);
          umma_ss<1>(d_o, pd + 16, vd + 128, idesc_o);
          umma_ss<1>(d_o, pd + 32, vd + 256, idesc_o);
          umma_ss<1>(d_o, pd + 48, vd + 384, idesc_o);
          mma_commit(&vo_empty[g & 1]);
        }
        __syncwarp();
        if (!warp_wait(&vp_full[g & 1], (g / 2) & 1, p.err, abort_flag)) return false;
        tc_fence_after();
        const uint64_t pd2 = noswz_desc(smem_u32(smem + OFF_P + (v ^ 1u) * P_BYTES), 128, 1024);
        const uint64_t vd2 = sw128_desc(smem_u32(v_peer), K_CHUNK, 1024);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i) umma_ss<1>(d_o, pd2 + 16 * i, vd2 + 128 * i, idesc_o);
          mma_commit(vp_empty);
          mma_commit_both(pv_done);
        }
        __syncwarp();
        return true;
      };
      Unit x;
      for (; ok && take_unit(ui, x);) {
        const int nsteps = (x.hi - x.lo + 2 * kTile - 1) / (2 * kTile);
        if (!(ok = warp_wait(q_full, ui & 1, p.err, abort_flag))) break;
        ++ui;
        if (nsteps == 0) {
          if (elect_one()) mma_commit(q_empty);
          __syncwarp();
        }
        for (int j = 0; j < nsteps; ++j, ++gi) {
          if (!(ok = warp_wait(&xy_full[gi & 1], (gi / 2) & 1, p.err, abort_flag))) break;
          if (gi >= 1 && !(ok = warp_wait(s_empty, (gi - 1) & 1, p.err, abort_flag))) break;
          tc_fence_after();
          const uint64_t vd = sw128_desc(smem_u32(v_own(gi)), 16, 1024);
          constexpr uint64_t kc = K_CHUNK >> 4, qc = Q_CHUNK >> 4;
          // place c of the block order, 16 dims (32 bytes, 8 tensor-memory columns) per product.  Loops over the blocks: the
          // hot code of all roles has to fit the instruction cache (all 36 products written out: 1110 -> 1138 us for 512
          // tokens at 16k context).
          if (elect_one()) {
#pragma unroll 1
            for (int c = 0; c < kSmemQ; ++c) {
              const uint64_t bd = c < kXBlocks ? xd + (uint64_t)c * kc : yd, ad = qd + (uint64_t)c * qc;
              umma_ss_acc(d_s, ad, bd, idesc_s, c > 0);
#pragma unroll
              for (int i = 1; i < 4; ++i) umma_ss<1>(d_s, ad + 2 * i, bd + 2 * i, idesc_s);
              if (c == kXBlocks - 1) mma_commit(x_empty);
            }
#pragma unroll 1
            for (int c = kSmemQ; c < kXBlocks + kYBlocks; ++c) {
              const uint64_t bd = yd + (uint64_t)(c - kXBlocks) * kc;
#pragma unroll
              for (int i = 0; i < 4; ++i) umma_ts<1>(d_s, a_q + (uint32_t)(32 * (c - kSmemQ) + 8 * i), bd + 2 * i, idesc_s);
            }
            mma_commit(y_empty);
          }
          __syncwarp();
          if (!(ok = warp_wait(&vo_full[gi & 1], (gi / 2) & 1, p.err, abort_flag))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll 2
            for (int c = kXBlocks + kYBlocks; c < kChunks; ++c) {
              const uint64_t bd = vd + (uint64_t)(c - kXBlocks - kYBlocks) * kc;
#pragma unroll
              for (int i = 0; i < 4; ++i) umma_ts<1>(d_s, a_q + (uint32_t)(32 * (c - kSmemQ) + 8 * i), bd + 2 * i, idesc_s);
            }
            mma_commit(s_full);
            if (j == nsteps - 1) mma_commit(q_empty);
          }
          __syncwarp();
          if (j > 0 && !(ok = issue_pv(gi - 1, j == 1))) break;
        }
        if (ok && nsteps > 0) ok = issue_pv(gi - 1, nsteps == 1);
      }
      if (elect_one()) mma_commit(fin);
      __syncwarp();
      mbar_wait(fin, 0, p.err, nullptr);
    } else if (warp == kLookupWarp) {
      // ------------------------------------------------------------------ units and pages, steps ahead
      int gi = 0;
      bool ok = true;
      int u = blockIdx.x / 2, nm = 0;
      for (int k = 0; ok; ++k) {
        Unit x;
        x.rows = -1;
        if (!p.next || k == 0) {  // both CTAs find it alike
          for (; u < units; u += clusters) {
            x = get_unit<kSrc>(p, 2 * u + (int)v, lane == 0 && v == 0 ? p.err : nullptr);
            if (x.rows > 0) break;
            x.rows = -1;
            if (p.next) break;
          }
        }
        if (p.next && x.rows < 0) {  // the next one nobody has: CTA 0 finds it and says so
          if (v == 0) {
            while (true) {
              int n = 0;
              if (lane == 0) n = clusters + atomicAdd(p.next, 1);
              u = __shfl_sync(0xFFFFFFFFu, n, 0);
              if (u >= units) break;
              x = get_unit<kSrc>(p, 2 * u, lane == 0 ? p.err : nullptr);
              if (x.rows > 0) break;
            }
            if (u >= units) x.rows = -1;
            if (lane == 0) st_async4(peer_address(smem + OFF_MAIL + (nm % 4) * 4, 1), (uint32_t)u, peer_address(&mail[nm % 4], 1));
          } else {
            if (lane == 0) mbar_arrive_expect_tx(&mail[nm % 4], 4);
            __syncwarp();
            if (!(ok = cluster_wait(&mail[nm % 4], (nm / 4) & 1, p.err, abort_flag))) break;
            u = *reinterpret_cast<volatile int*>(smem + OFF_MAIL + (nm % 4) * 4);
            if (u < units) x = get_unit<kSrc>(p, 2 * u + 1, nullptr);
          }
          ++nm;
        }
        if (k >= kUnitSlots && !(ok = warp_wait(&u_empty[k % kUnitSlots], ((k / kUnitSlots) - 1) & 1, p.err, abort_flag))) break;
        if (lane == 0) {
          unit_ring[k % kUnitSlots] = x;
          mbar_arrive(&u_full[k % kUnitSlots]);
        }
        if (x.rows < 0) break;
        const int32_t* table = p.block_table + (int64_t)max(0, x.req) * p.max_blocks;
        const int nsteps = (x.hi - x.lo + 2 * kTile - 1) / (2 * kTile);
        if constexpr (kQuant) {
          // lane: keys lane and lane + 32 of the own page and of the other; selected positions are loaded a step ahead
          auto position = [&](int j, int e) -> int {
            const int slot = x.lo + (2 * j + (e < 2 ? (int)v : 1 - (int)v)) * kTile + lane + 32 * (e & 1);
            if (slot >= x.hi) return -1;
            return kSrc == kSelected && p.idx ? p.idx[(int64_t)(x.row0 / p.H) * p.k + slot] : slot;
          };
          int ps[4], next[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) ps[e] = position(0, e);
          for (int j = 0; j < nsteps; ++j, ++gi) {
            int row[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) next[e] = position(j + 1, e);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool seen = x.req >= 0 && ps[e] >= 0 && (kSrc != kSelected || ps[e] <= x.tok0);
              row[e] = seen && ps[e] / kTile < p.max_blocks ? table[ps[e] / kTile] : -1;
              if (seen && (row[e] < 0 || row[e] >= p.num_blocks)) {
                if (e < 2) raise_error(p.err, DSA_DEVERR_BLOCK_ID);
                row[e] = -1;
              }
              if (row[e] >= 0) row[e] = row[e] * kTile + ps[e] % kTile;
              if (kSrc == kSelected && e < 2 && !seen && ps[e] != -1 && x.req >= 0) raise_error(p.err, DSA_DEVERR_INDEX);
            }
            if (gi >= kSlots && !(ok = warp_wait(&r_empty[gi % kSlots], ((gi / kSlots) - 1) & 1, p.err, abort_flag))) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) row_ring[(gi % kSlots * 2 + (e >> 1)) * kTile + lane + 32 * (e & 1)] = row[e];
            __syncwarp();
            if (lane == 0) mbar_arrive(&r_full[gi % kSlots]);
#pragma unroll
            for (int e = 0; e < 4; ++e) ps[e] = next[e];
          }
        } else
        for (int j = 0; j < nsteps; ++j, ++gi) {
          int page[2];
          uint32_t may[2][2];
#pragma unroll
          for (int w = 0; w < 2; ++w) {  // own page, the other
            const int base = x.lo + (2 * j + (w ? 1 - (int)v : (int)v)) * kTile, lblk = base / kTile;
            page[w] = -1;
            may[w][0] = may[w][1] = ~0u;
            if (base >= x.hi) continue;
            page[w] = lblk < p.max_blocks ? table[lblk] : -1;
            if (page[w] < 0 || page[w] >= p.num_blocks) {
              raise_error(p.err, DSA_DEVERR_BLOCK_ID);
              page[w] = -1;
            }
            if (p.linear_pages && page[w] >= 0) {
              page[w] = x.req * p.linear_pages + lblk;
              const uint8_t* f = p.row_ok + (int64_t)page[w] * kTile;
              may[w][0] = __ballot_sync(0xFFFFFFFFu, f[lane] != 0);
              may[w][1] = __ballot_sync(0xFFFFFFFFu, f[lane + 32] != 0);
            }
          }
          if (gi >= kSlots && !(ok = warp_wait(&r_empty[gi % kSlots], ((gi / kSlots) - 1) & 1, p.err, abort_flag))) break;
          if (lane == 0) {
            int4* e = reinterpret_cast<int4*>(row_ring + gi % kSlots * 8);
            e[0] = make_int4(page[0], page[1], (int)may[0][0], (int)may[0][1]);
            e[1] = make_int4((int)may[1][0], (int)may[1][1], 0, 0);
            mbar_arrive(&r_full[gi % kSlots]);
          }
        }
        if (!ok) break;
        u += clusters;
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (*abort_flag) {  // gave up: what is on its way to the other CTA gets a millisecond to arrive
    for (const long long t0 = clock64(); clock64() - t0 < 2000000LL;) {
    }
  }
  cluster_sync_all();  // nothing of the other CTA is on its way here any more
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

}  // namespace

template <Source kSrc>
cudaError_t packed::launch_pair(const Params& p, const CUtensorMap& qmap, const CUtensorMap& rmap, const CUtensorMap& pmap, int num_sms,
                                cudaStream_t s) {
  auto kernel = mla_pair_kernel<kSrc>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  const int units = p.tiles * p.nsplit, pairs = num_sms / 2;
  cudaLaunchAttribute attrs[2];
  const cudaLaunchConfig_t cfg = launch_config(dim3(2 * (units < pairs ? units : pairs)), dim3(kThreads), SMEM, s, attrs, 2);
  return cudaLaunchKernelEx(&cfg, kernel, qmap, rmap, pmap, p);
}
template cudaError_t packed::launch_pair<kSelected>(const Params&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
template cudaError_t packed::launch_pair<kPages>(const Params&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
template cudaError_t packed::launch_pair<kPagesBf16>(const Params&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);

}  // namespace dsa
