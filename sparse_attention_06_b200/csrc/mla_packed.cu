// mla_packed.cu -- MLA (MQA mode) for tiles of 128 query rows on tcgen05 tensor cores: dense attention of
// chunks over the paged latent cache, and sparse attention over quantised latents.
//
// Mathematics: out = softmax(tau Q K^T + mask) V with K the 576-wide latent rows and V their first
// 512 elements, by one pass over the keys with a running maximum and sum per query row.
//
// Query rows.  A token's H heads are H rows of the [num_tokens * H, 576] query matrix and a chunk's
// tokens follow each other, so 128 consecutive rows of that matrix are one tensor-core tile whatever H
// is: with 16 heads a tile holds eight tokens of the request, which share every key tile.  Row r of a
// tile belongs to token (first row + r) / H of the chunk; the causal mask is the only thing that
// differs between the tokens of a tile.  (Sparse attention: one query per tile, its keys are its own.)
//
// Work unit = (row tile, key split sp, value half v), as in the bf16 sparse kernel: O of 128 rows x
// 512 values in f32 would fill tensor memory, so two CTAs take 256 values each and both compute S.
// Per 64-key tile: S = Q K^T (M = 128, N = 64, K = 576), softmax, O_v += P V_v (N = 256, K = 64).
// Tensor memory: O_v [0, 256), S [256, 320), six of Q's nine 64-dim column blocks [320, 512).  Shared
// memory: the other three (48 KB), P (16 KB), and the key tile as bf16 in 64-row x 64-dim blocks of 8 KB
// (128B-swizzled: K-major B of Q K^T and, for the value blocks, MN-major B of P V at once).
//
// A tile's nine blocks live in three rings, by how long each is needed: the four blocks of this
// CTA's values until P V is done (three stages), the other blocks only until Q K^T is (three blocks
// with two stages, two blocks - the first that Q K^T reads - with one).  So the tensor core can run Q K^T of
// tile g + 1, P V of tile g and the filling of tile g + 2 at once in 160 KB; whole tiles of 72 KB would
// leave room for two stages, each held from the first load to the end of P V.
//
// Quantised latents become bf16 on their way in: eight warps load a row's 512 codes with
// 16-byte loads (one tile ahead, into registers), turn them into bf16 (exact: a code has four
// significant bits and its scale is a power of two) and store them in the swizzled layout.  bf16
// latents come by TMA: whole 64-token pages as nine 64-row boxes, a page's visible part by gather4.
//
// Roles (16 warps): 0-7 fill the rings and move Q into tensor memory (staged by TMA through idle
// ring blocks at the start of a unit); 8-11 softmax and epilogue, one row per thread; 12 issues the
// products (the whole warp, so that the compiler keeps the issue uniform: with elect.sync one M = 128, N = 64
// product is issued every ~32 cycles, against ~60 from a thread chosen by its index); 13 looks the
// keys' pool rows up, a few tiles ahead.
// All waits are bounded; bad rows set the device error word and are skipped.
#include "mla_packed.cuh"

namespace dsa {
namespace {

using namespace packed;

constexpr int kYStages = 2, kVStages = 3;
constexpr int OFF_Q = 0;
constexpr int OFF_P = OFF_Q + kSmemQ * Q_CHUNK;
constexpr int OFF_Y = OFF_P + kRows * kTile * 2;
constexpr int OFF_X = OFF_Y + kYStages * kYBlocks * K_CHUNK;
constexpr int OFF_V = OFF_X + kXBlocks * K_CHUNK;
constexpr int OFF_BAR = OFF_V + kVStages * kVBlocks * K_CHUNK;
constexpr int NBAR = 36;
constexpr int kMaskSlots = 4;
constexpr int kMaskBytes = 8;                            // of a slot: one byte per fill warp, a bit per key
constexpr int OFF_MASK = OFF_BAR + NBAR * 8;             // [slot] keys with a row to see
constexpr int OFF_POISON = OFF_MASK + kMaskSlots * kMaskBytes;  // [slot] rows with NaN or infinity, see below
constexpr int kRowSlots = 4;
constexpr int OFF_STATS = OFF_POISON + kMaskSlots * kMaskBytes;   // 1 / l of each row (last unit)
constexpr int OFF_MISC = OFF_STATS + kRows * 4;
constexpr int OFF_UNIT = OFF_MISC + 16;                  // [2] units in hand
constexpr int OFF_ROWS = OFF_UNIT + 2 * 40;                  // quantised: [slot][64] pool row of each key of a tile, -1: none to see;
                                                         // bf16: [slot] page of the tile and its rows that may be read,
                                                         // then [2][2][128] row maxima exchanged
constexpr int SMEM = OFF_ROWS + kRowSlots * 16 + 2 * 2 * kRows * 4;
static_assert(kRowSlots * kTile * 4 <= 2 * 2 * kRows * 4, "row ring");
static_assert(SMEM <= 232448, "shared memory budget");
static_assert(kYStages * kYBlocks * K_CHUNK == 3 * Q_CHUNK && kXBlocks * K_CHUNK == Q_CHUNK && kVBlocks * K_CHUNK == 2 * Q_CHUNK,
              "six Q blocks are staged in the Y and X rings and one V stage");

// Warps by source: 0-7 fill; softmax, `kParts` warps per 32 rows (bf16 tiles come fast enough that one warp's
// softmax, a chain of ~2100 cycles, would set the pace); one to issue products, one to look pages up, two idle
// ones to complete the warpgroup.  Registers a thread by warpgroup, within what the block was launched with:
// quantised 2 x 136 + 136 + 104 = 4 x 128, bf16 2 x 80 + 2 x 104 + 104 <= 5 x 96.  (Spilled registers cost more than
// elsewhere: they miss the small L1 left beside 227 KB of shared memory.)
template <Source kSrc>
struct Roles {
  static constexpr bool kQuant = kSrc != kPagesBf16;
  static constexpr int kParts = kQuant ? 1 : 2;
  static constexpr int kSoftmaxWarp = kFillWarps, kIssueWarp = kFillWarps + 4 * kParts, kLookupWarp = kIssueWarp + 1;
  static constexpr int kThreads = 32 * (kIssueWarp + 4);
  static constexpr int kFillRegs = kQuant ? 136 : 80, kSoftmaxRegs = kQuant ? 136 : 104, kIssueRegs = 104;
};

template <Source kSrc>
__global__ void __launch_bounds__(Roles<kSrc>::kThreads, 1)
    mla_packed_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap rmap,
                      const __grid_constant__ CUtensorMap pmap, const Params p) {
  using R = Roles<kSrc>;
  constexpr bool kQuant = R::kQuant;
  constexpr int kParts = R::kParts, kIssueWarp = R::kIssueWarp;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // (swizzled blocks need it; the whole of shared memory starts there)
    if (threadIdx.x == 0) raise_error(p.err, DSA_DEVERR_TIMEOUT);
    return;
  }
  uint8_t* q_s = smem + OFF_Q;
  uint8_t* p_s = smem + OFF_P;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* k_full = bars + 0;      // [2] rows of the tile in place, masks published
  uint64_t* land = bars + 2;        // [2] bf16 rows landed, to be looked over before k_full
  uint64_t* x_empty = bars + 4;     // Q K^T is past the tile's X blocks
  uint64_t* y_empty = bars + 5;     // [kYStages] ... past its Y blocks
  uint64_t* v_empty = bars + 7;     // [kVStages] P V done
  uint64_t* q_stage = bars + 10;    // the unit's Q landed (staged blocks and shared-memory part)
  uint64_t* q_read = bars + 11;     // staged Q read: the ring blocks may be filled
  uint64_t* q_full = bars + 12;     // Q of the unit in place
  uint64_t* q_empty = bars + 13;    // the unit's last Q K^T has completed
  uint64_t* s_full = bars + 14;
  uint64_t* s_empty = bars + 15;
  uint64_t* p_full = bars + 16;
  uint64_t* pv_done = bars + 17;
  uint64_t* fin = bars + 18;        // every product has completed
  uint64_t* ep_last = bars + 19;    // last unit: 1 / l published after its last P V
  uint64_t* r_full = bars + 20;     // [kRowSlots] pool rows of a tile looked up
  uint64_t* r_empty = bars + 24;    // [kRowSlots] ... read by the fill warps
  uint8_t* masks = smem + OFF_MASK;
  int32_t* row_ring = reinterpret_cast<int32_t*>(smem + OFF_ROWS);
  float* row_max = reinterpret_cast<float*>(smem + OFF_ROWS + kRowSlots * 16);
  uint64_t* u_full = bars + 32;     // [kUnitSlots] a unit (or the end) published
  uint64_t* u_empty = bars + 34;    // [kUnitSlots] ... taken by every warp that works on it
  Unit* unit_ring = reinterpret_cast<Unit*>(smem + OFF_UNIT);
  uint64_t* x_bar = bars + 28;      // [4] the two softmax warps of 32 rows have exchanged their maxima
  uint8_t* poisons = smem + OFF_POISON;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 8);
  float* stats = reinterpret_cast<float*>(smem + OFF_STATS);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = p.tiles * p.nsplit * 2;
  griddep_launch_dependents();

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], kFillWarps);
      mbar_init(&land[i], kFillWarps);
    }
    for (int i = 0; i < kRowSlots; ++i) {
      mbar_init(&r_full[i], 1);
      mbar_init(&r_empty[i], kFillWarps);
    }
    mbar_init(x_empty, 1);
    for (int i = 0; i < kYStages; ++i) mbar_init(&y_empty[i], 1);
    for (int i = 0; i < kVStages; ++i) mbar_init(&v_empty[i], 1);
    mbar_init(q_stage, 1);
    mbar_init(q_read, kFillWarps);
    mbar_init(q_full, kFillWarps);
    mbar_init(q_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(s_empty, 4 * kParts);
    mbar_init(p_full, 4 * kParts);
    mbar_init(pv_done, 1);
    mbar_init(fin, 1);
    mbar_init(ep_last, 128 * kParts);
    for (int i = 0; i < 4; ++i) mbar_init(&x_bar[i], 2);
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
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();

  // unit number k of this CTA (the lookup warp publishes it; false: none, or gave up)
  auto take_unit = [&](int k, Unit& x) -> bool {
    if (!warp_wait(&u_full[k % kUnitSlots], (k / kUnitSlots) & 1, p.err, abort_flag)) return false;
    x = unit_ring[k % kUnitSlots];
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_empty[k % kUnitSlots]);
    return x.rows > 0;
  };
  // whether unit k is the CTA's last (asked when its work is done, so that the next is known)
  auto last_unit = [&](int k, bool& last) -> bool {
    if (!warp_wait(&u_full[(k + 1) % kUnitSlots], ((k + 1) / kUnitSlots) & 1, p.err, abort_flag)) return false;
    last = unit_ring[(k + 1) % kUnitSlots].rows < 0;
    return true;
  };

  if (warp < kFillWarps) {
    if constexpr (kQuant)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kFillRegs));
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kFillRegs));
    // ------------------------------------------------------------------ rings and Q
    const int quarter = warp & 3, part = warp >> 2;
    const uint32_t my_lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const int half = (lane >> 2) & 1, l16 = (lane & 3) | (lane >> 3) << 2;  // quantised rows: two at a time, 16 lanes each
    int gi = 0, ui = 0;
    uint32_t nland[2] = {0u, 0u};
    bool ok = true, staged = false;
    Unit x;
    for (; ok && take_unit(ui, x);) {
      const int ntiles = (x.hi - x.lo + kTile - 1) / kTile;
      const bool report = x.v == 0;

      // pool row of key `key` of this warp's, of CTA tile g (r_full of that tile has been waited for)
      auto row_of = [&](int g, int key) -> int { return row_ring[g % kRowSlots * kTile + warp * kKeysPerWarp + key]; };
      auto wait_rows = [&](int g) { return warp_wait(&r_full[g % kRowSlots], (g / kRowSlots) & 1, p.err, abort_flag); };

      // --- quantised rows in flight: pair q is the warp's keys 2 q + half; a lane has 16 codes of its row in
      // this CTA's value half (hh = 0) and 16 in the other (hh = 1).  Lane l has the scale of key l / 4 % 4, group
      // l % 4.  Loads of one kind are issued together, as far as possible ahead of
      // their use: a warp waits for loads by a handful of counters, so waiting for an old load can mean waiting
      // for a young one that shares its counter.  None is conditional (a key without a row reads row 0).
      constexpr int kPairs = kKeysPerWarp / 2;
      constexpr uint32_t kAll = (1u << kKeysPerWarp) - 1u;
      uint4 code[kPairs][2];
      float sc = 1.0f;
      uint32_t seen = 0u, bad = 0u;  // of the tile in registers: keys with a row; lanes with no row or no power of two
      auto load_codes = [&](int g, int hh) {
        const uint8_t* base = p.data + 256 * (hh ^ x.v) + 16 * l16;
#pragma unroll
        for (int q = 0; q < kPairs; ++q) code[q][hh] = load16_here(base + (int64_t)max(0, row_of(g, 2 * q + half)) * kLatentBytes);
      };
      auto load_scales = [&](int g) -> float { return loadf_here(p.scale + (int64_t)max(0, row_of(g, (lane >> 2) & (kKeysPerWarp - 1))) * 4 + (lane & 3)); };
      auto check_rows = [&](int g) {
        const bool none = row_of(g, (lane >> 2) & (kKeysPerWarp - 1)) < 0;
        bad = __ballot_sync(0xFFFFFFFFu, none || !latent_scale_ok(sc));
        seen = ~__ballot_sync(0xFFFFFFFFu, none);
      };
      if (kQuant && ntiles > 0) {
        if (!(ok = wait_rows(gi))) break;
        sc = load_scales(gi);
        load_codes(gi, 0);
        load_codes(gi, 1);
        check_rows(gi);
      }

      // --- Q of the unit, once the unit before is past its last Q K^T: places 0 .. 2 of the order to
      // shared memory, 3 .. 8 through the idle Y and X rings and the V stage next in turn to tensor memory
      if (ui >= 1 && !(ok = warp_wait(q_empty, (ui - 1) & 1, p.err, abort_flag))) break;
      if (gi >= kVStages && !(ok = warp_wait(&v_empty[gi % kVStages], ((gi / kVStages) - 1) & 1, p.err, abort_flag))) break;
      uint8_t* v_stage0 = smem + OFF_V + gi % kVStages * kVBlocks * K_CHUNK;
      if (tid == 0) {
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(q_stage, kChunks * Q_CHUNK);
        for (int c = kSmemQ; c < kChunks; ++c) {
          const int b = c - kSmemQ;
          tma_load_2d(b < 4 ? smem + OFF_Y + b * Q_CHUNK : v_stage0 + (b - 4) * Q_CHUNK, &qmap, q_stage, block_of(c, x.v) * 64, x.row0);
        }
        for (int c = 0; c < kSmemQ; ++c) tma_load_2d(q_s + c * Q_CHUNK, &qmap, q_stage, block_of(c, x.v) * 64, x.row0);
        staged = true;
      }
      tc_fence_after();
      if (!(ok = warp_wait(q_stage, ui & 1, p.err, abort_flag))) break;
      staged = false;
      {
        const int r = quarter * 32 + lane;
#pragma unroll
        for (int b = 0; b < 6; ++b) {  // this warp's half (64 bytes) of the row's block
          const uint8_t* src = (b < 4 ? smem + OFF_Y + b * Q_CHUNK : v_stage0 + (b - 4) * Q_CHUNK) + r * 128;
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

      // --- the unit's key tiles
      for (int j = 0; j < ntiles; ++j, ++gi) {
        const int s = gi & 1, slot = gi % kMaskSlots;
        uint8_t* v_st = smem + OFF_V + gi % kVStages * kVBlocks * K_CHUNK;
        uint8_t* y_st = smem + OFF_Y + gi % kYStages * kYBlocks * K_CHUNK;
        uint8_t* x_st = smem + OFF_X;
        auto wait_v = [&]() { return gi < kVStages || warp_wait(&v_empty[gi % kVStages], ((gi / kVStages) - 1) & 1, p.err, abort_flag); };
        auto wait_y = [&]() { return gi < kYStages || warp_wait(&y_empty[gi % kYStages], ((gi / kYStages) - 1) & 1, p.err, abort_flag); };
        auto wait_x = [&]() { return gi < 1 || warp_wait(x_empty, (gi - 1) & 1, p.err, abort_flag); };
        if constexpr (kQuant) {
          // rows that only some of the tile's tokens see: a NaN there must not reach the others through 0 * NaN
          // in P V, so it becomes zero and its row is noted: the softmax makes the weights of the tokens that see
          // it NaN (elsewhere a NaN takes its natural course)
          const bool partly = kSrc != kSelected && x.lo + j * kTile + kTile - 1 > x.tok0 && x.hi - 1 > x.tok0;
          uint32_t nan_rows = 0u;
          // 16 codes into the row's blocks: `dst` is the row of the lane's 64-dim block, pieces 2 (l16 % 4) and
          // the next; eight consecutive lanes hold four pieces of both rows of a pair, which differ in bit 0, so
          // they store to all eight bank groups.  kPlain: every key has a row, and all tokens see them.
          auto put = [&](auto plain, int q, int hh, uint8_t* dst) {
            constexpr bool kPlain = decltype(plain)::value;
            const int r = warp * kKeysPerWarp + 2 * q + half;
            uint32_t w[4] = {code[q][hh].x, code[q][hh].y, code[q][hh].z, code[q][hh].w};
            float my_sc = __shfl_sync(0xFFFFFFFFu, sc, (2 * q + half) * 4 + 2 * (hh ^ x.v) + (l16 >> 3));
            if (!kPlain && ((bad >> (4 * (2 * q + half))) & 0xFu)) {
              w[0] = w[1] = w[2] = w[3] = 0u;
              my_sc = 1.0f;
            }
            uint32_t b[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) decode4(w[i], make_float2(my_sc, my_sc), b[2 * i], b[2 * i + 1]);
            if (!kPlain && partly) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if ((b[i] & 0x7F80u) == 0x7F80u) { b[i] &= 0xFFFF0000u; nan_rows |= 1u << (2 * q + half); }
                if ((b[i] & 0x7F800000u) == 0x7F800000u) { b[i] &= 0xFFFFu; nan_rows |= 1u << (2 * q + half); }
              }
            }
            const uint32_t piece = (uint32_t)(l16 & 3) * 2u, x7 = (uint32_t)(r & 7);
            *reinterpret_cast<uint4*>(dst + r * 128 + ((piece ^ x7) << 4)) = make_uint4(b[0], b[1], b[2], b[3]);
            *reinterpret_cast<uint4*>(dst + r * 128 + (((piece + 1u) ^ x7) << 4)) = make_uint4(b[4], b[5], b[6], b[7]);
          };
          auto put_all = [&](int hh, uint8_t* dst) {
            if (bad == 0u && !partly) {
#pragma unroll
              for (int q = 0; q < kPairs; ++q) put(Flag<true>(), q, hh, dst);
            } else {
#pragma unroll
              for (int q = 0; q < kPairs; ++q) put(Flag<false>(), q, hh, dst);
            }
          };
          if (!(ok = wait_v())) break;
          put_all(0, v_st + (l16 >> 2) * K_CHUNK);
          const bool more = j + 1 < ntiles;
          float sc_n = 1.0f;
          if (more) {
            if (!(ok = wait_rows(gi + 1))) break;
            sc_n = load_scales(gi + 1);
            load_codes(gi + 1, 0);
          }
          if (!(ok = wait_y()) || !(ok = wait_x())) break;
          // the RoPE part as it is, in the background (zeros for a row that is not there)
#pragma unroll
          for (int i = 0; i < kKeysPerWarp / 4; ++i) {
            const int r8 = 4 * i + (lane >> 3);
            const int r = warp * kKeysPerWarp + r8;
            cp_async_16(smem_u32(x_st + r * 128 + (((lane & 7) ^ (r & 7)) << 4)),
                        p.data + (int64_t)max(0, row_of(gi, r8)) * kLatentBytes + kDv + 16 * (lane & 7),
                        ((bad >> (4 * r8)) & 0xFu) ? 0u : 16u);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&r_empty[gi % kRowSlots]);
          put_all(1, (l16 >> 2) == 3 ? x_st + K_CHUNK : y_st + (l16 >> 2) * K_CHUNK);
          const uint32_t poison = __reduce_or_sync(0xFFFFFFFFu, nan_rows);
          if (lane == 0) {
            uint32_t valid = kAll;
            if (bad) {
              bool flag = false;
              for (int r8 = 0; r8 < kKeysPerWarp; ++r8)
                if ((bad >> (4 * r8)) & 0xFu) {
                  valid &= ~(1u << r8);
                  flag |= (seen >> (4 * r8)) & 1u;
                }
              if (report && flag) raise_error(p.err, DSA_DEVERR_SCALE);
            }
            masks[slot * kMaskBytes + warp] = (uint8_t)valid;
            poisons[slot * kMaskBytes + warp] = (uint8_t)(poison & valid);
          }
          if (more) {
            sc = sc_n;
            check_rows(gi + 1);
            load_codes(gi + 1, 1);
          }
          cp_async_wait_all();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[s]);
        } else {
          if (!(ok = wait_rows(gi))) break;
          const int page = row_ring[gi % kRowSlots * 4], key = warp * kKeysPerWarp + (lane & 7);
          const bool may = ((uint32_t)row_ring[gi % kRowSlots * 4 + 2 + (key >> 5)] >> (key & 31)) & 1u;
          const int row = page >= 0 && may && x.lo + j * kTile + key < x.hi ? page * kTile + key : -1;
          const uint32_t valid = __ballot_sync(0xFFFFFFFFu, row >= 0) & 0xFFu;
          if (lane == 0) mbar_arrive(&r_empty[gi % kRowSlots]);
          const int base = x.lo + j * kTile;
          const bool whole = base + kTile <= x.hi && valid == 0xFFu;
          // (as above; these rows are looked over once they have landed)
          const bool partly = base + kTile - 1 > x.tok0 && x.hi - 1 > x.tok0;
          uint64_t* bar = partly ? &land[s] : &k_full[s];
          // this warp's eight rows (or, for a whole page, warp 0 all of them): places lo .. hi - 1 of the order
          auto copy = [&](int lo, int hi, uint8_t* dst) {
            if (whole) {
              if (warp == 0 && lane == 0)
                for (int c = lo; c < hi; ++c) tma_load_2d(dst + (c - lo) * K_CHUNK, &pmap, bar, block_of(c, x.v) * 64, page * kTile);
              return;
            }
#pragma unroll
            for (int g4 = 0; g4 < 2; ++g4) {
              const int rc = row >= 0 ? row : p.oob_row;
              const int r0 = __shfl_sync(0xFFFFFFFFu, rc, 4 * g4), r1 = __shfl_sync(0xFFFFFFFFu, rc, 4 * g4 + 1);
              const int r2 = __shfl_sync(0xFFFFFFFFu, rc, 4 * g4 + 2), r3 = __shfl_sync(0xFFFFFFFFu, rc, 4 * g4 + 3);
              if (lane == 0)
                for (int c = lo; c < hi; ++c)
                  tma_gather4(dst + (c - lo) * K_CHUNK + (warp * kKeysPerWarp + 4 * g4) * 128, &rmap, bar, block_of(c, x.v) * 64, r0, r1, r2, r3);
            }
          };
          if (!(ok = wait_y())) break;
          if (lane == 0) {
            masks[slot * kMaskBytes + warp] = (uint8_t)valid;
            if (!partly) poisons[slot * kMaskBytes + warp] = 0;
            fence_proxy_async_smem();
            if (!whole)
              mbar_arrive_expect_tx(bar, kKeysPerWarp * kDqk * 2);
            else if (warp == 0)
              mbar_arrive_expect_tx(bar, K_BYTES);
            else
              mbar_arrive(bar);
          }
          __syncwarp();
          copy(2, 5, y_st);
          if (!(ok = wait_v())) break;
          copy(5, 9, v_st);
          if (!(ok = wait_x())) break;
          copy(0, 2, x_st);
          if (partly) {
            if (!(ok = warp_wait(&land[s], nland[s] & 1, p.err, abort_flag))) break;
            ++nland[s];
            // values that are not finite become zero and their row is noted: the softmax makes the weights
            // of the tokens that see it NaN, the others' products stay as they are.  (The V ring is all that
            // P V reads; a NaN in the other blocks only reaches logits, of hidden keys masked ones.)
            uint32_t poison = 0u;
            for (int r8 = 0; r8 < kKeysPerWarp; ++r8) {
              const int r = warp * kKeysPerWarp + r8;
              if (base + r <= x.tok0 || base + r >= x.hi) continue;
              // 32 pieces of 16 bytes: the row's 256 values of this half
              uint4* at = reinterpret_cast<uint4*>(v_st + (lane >> 3) * K_CHUNK + r * 128 + ((lane & 7) << 4));
              const uint4 y = *at;
              uint32_t w[4] = {y.x, y.y, y.z, y.w};
              bool f = false;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((w[k] & 0x7F80u) == 0x7F80u) { w[k] &= 0xFFFF0000u; f = true; }
                if ((w[k] & 0x7F800000u) == 0x7F800000u) { w[k] &= 0xFFFFu; f = true; }
              }
              if (f) *at = make_uint4(w[0], w[1], w[2], w[3]);
              if (__any_sync(0xFFFFFFFFu, f)) poison |= 1u << r8;
            }
            if (lane == 0) poisons[slot * kMaskBytes + warp] = (uint8_t)poison;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_full[s]);
          }
        }
      }
      if (!ok) break;
      bool last;
      if (!(ok = last_unit(ui - 1, last))) break;
      if (last) {
        // the CTA's last unit: these warps store part of O_v / l too, staged in the V ring (free after the last P V)
        if (!(ok = warp_wait(ep_last, 0, p.err, abort_flag))) break;
        tc_fence_after();
        // (of the 256 columns 64 are each softmax warp's)
        const int width = kParts == 2 ? 64 : 96, lo = 64 + (kParts == 2 ? 128 : 96) * part;
        store_o(p, x, my_lanes, quarter, lo, lo + width, smem + OFF_V + warp * 2048,
                stats[quarter * 32 + lane], ntiles > 0);
        tc_fence_before();
      }
    }
    // gave up: copies in flight must land before the CTA exits
    if (!ok && staged) mbar_wait(q_stage, ui & 1, p.err, nullptr);
    if (!ok && !kQuant && lane == 0) {
      for (int t = gi - 1; t <= gi; ++t)
        if (t >= 0) mbar_wait(&k_full[t & 1], (uint32_t)((t / 2) & 1), p.err, nullptr);
      for (int i = 0; i < 2; ++i) mbar_wait(&land[i], nland[i] & 1, p.err, nullptr);
    }
  } else if (warp < kIssueWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kSoftmaxRegs));
    // ------------------------------------------------------------------ softmax and epilogue
    constexpr int kCols = kTile / kParts;  // keys of a tile, and columns of O_v in kHalf / kParts, of one warp
    const int quarter = warp & 3, part = (warp - R::kSoftmaxWarp) >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    int gi = 0, nx = 0;
    bool ok = true;
    // both parts' values of this row, combined by f (a bounded wait for the other warp)
    auto exchange = [&](float mine, float& other) -> bool {
      float* buf = row_max + (nx & 1) * 2 * kRows;
      buf[part * kRows + r] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(&x_bar[quarter]);
      if (!warp_wait(&x_bar[quarter], nx & 1, p.err, abort_flag)) return false;
      ++nx;
      other = buf[(1 - part) * kRows + r];
      return true;
    };
    Unit x;
    for (int ui = 0; ok && take_unit(ui, x); ++ui) {
      const int ntiles = (x.hi - x.lo + kTile - 1) / kTile;
      // last position this row sees (kSelected: the tile's own mask tells)
      int limit;
      if constexpr (kSrc == kSelected)
        limit = r < x.rows ? 0x7FFFFFFF : -1;
      else
        limit = r < x.rows ? x.tok0 + (x.h0 + r) / p.H : -1;
      float m_used = -INFINITY, l = 0.0f;
      for (int j = 0; j < ntiles; ++j, ++gi) {
        const int slot = gi % kMaskSlots;
        if (!(ok = warp_wait(s_full, gi & 1, p.err, abort_flag))) break;
        if (!(ok = warp_wait(&k_full[gi & 1], (gi / 2) & 1, p.err, abort_flag))) break;  // (long past: orders the masks)
        tc_fence_after();
        uint32_t sv[kCols];
#pragma unroll
        for (int c = 0; c < kCols / 16; ++c)
          tmem_ld16(lane_base + TM_S + part * kCols + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&sv[16 * c]));
        uint64_t valid = *reinterpret_cast<const volatile uint64_t*>(masks + slot * kMaskBytes);
        uint64_t poison = *reinterpret_cast<const volatile uint64_t*>(poisons + slot * kMaskBytes);
        const int d = limit - (x.lo + j * kTile);  // this row sees the tile's keys 0 .. d
        if (d < 63) valid &= d < 0 ? 0ull : (2ull << d) - 1ull;
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty);
        if (!__all_sync(0xFFFFFFFFu, valid == ~0ull && poison == 0ull)) {
          valid >>= part * kCols;
          poison >>= part * kCols;
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            if ((poison >> c) & 1u) sv[c] = 0x7FC00000u;
            if (!((valid >> c) & 1u)) sv[c] = 0xFF800000u;
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(sv[c]);
#pragma unroll
        for (int c = 4; c < kCols; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(sv[c]));
        float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        if constexpr (kParts == 2) {
          float other;
          if (!(ok = exchange(mt, other))) break;
          mt = fmaxf(mt, other);
        }
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
        uint32_t pk[kCols / 2];
        const float nsub = m_used == -INFINITY ? 0.0f : -m_used;
        float2 ps[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), ns2 = make_float2(nsub, nsub);
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
          const float2 e = fma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sc2, ns2);
          const float2 w = make_float2(fast_exp2(e.x), fast_exp2(e.y));
          // (the normaliser sums the weights before their rounding to bf16, which P V needs)
          ps[(c >> 1) & 1] = add2(ps[(c >> 1) & 1], w);
          const __nv_bfloat162 b = __floats2bfloat162_rn(w.x, w.y);
          pk[c >> 1] = *reinterpret_cast<const uint32_t*>(&b);
        }
        const float2 pt = add2(ps[0], ps[1]);
        l += pt.x + pt.y;
        // O and the P buffer are free once the previous tile's P V has completed
        if (gi >= 1 && !(ok = warp_wait(pv_done, (gi - 1) & 1, p.err, abort_flag))) break;
        if (rescale && j > 0) {
          tc_fence_after();
#pragma unroll 1
          for (int c0 = part * (kHalf / kParts); c0 < (part + 1) * (kHalf / kParts); c0 += 32) {
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
        uint8_t* prow = p_s + (r >> 3) * 1024 + (r & 7) * 16 + part * (kCols / 8) * 128;
#pragma unroll
        for (int kc = 0; kc < kCols / 8; ++kc)
          *reinterpret_cast<uint4*>(prow + kc * 128) = make_uint4(pk[4 * kc], pk[4 * kc + 1], pk[4 * kc + 2], pk[4 * kc + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (!ok) break;
      if constexpr (kParts == 2) {
        float other;
        if (!(ok = exchange(l, other))) break;
        l = part ? other + l : l + other;
      }
      if (ntiles > 0 && !(ok = warp_wait(pv_done, (gi - 1) & 1, p.err, abort_flag))) break;
      tc_fence_after();
      // a row that saw nothing: 0 and -inf; NaN stays NaN
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const float lse = l == 0.0f ? -INFINITY : (m_used + log2f(l)) * 0.69314718055994531f;
      bool last;
      if (!(ok = last_unit(ui, last))) break;
      if (last) {
        if (part == 0) stats[r] = inv;
        mbar_arrive(ep_last);
      }
      const int lo = part * (kHalf / 2);
      store_o(p, x, lane_base, quarter, lo, last ? lo + 64 : lo + kHalf / kParts, p_s + (warp - R::kSoftmaxWarp) * 2048, inv, ntiles > 0);
      if (x.v == 0 && part == 0 && r < x.rows) {
        if (x.splits == 1) {
          if (p.lse) p.lse[(int64_t)x.row0 + r] = lse;
        } else {
          p.part_lse[(int64_t)x.prow + r] = lse;
        }
      }
      tc_fence_before();
    }
  } else {
    if constexpr (kQuant)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kIssueRegs));
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kIssueRegs));
    if (warp == kIssueWarp) {
      // ------------------------------------------------------------------ the products
      // Order: Q K^T of tile g, then P V of tile g - 1.  So while the softmax reads S of tile g the tensor
      // core works on P V, and it never idles for S's only buffer.
      const uint32_t idesc_s = idesc_f16(1u, 0u, (uint32_t)kRows, (uint32_t)kTile);
      const uint32_t idesc_o = idesc_f16(1u, 1u, (uint32_t)kRows, (uint32_t)kHalf);
      const uint64_t qd = sw128_desc(smem_u32(q_s), 16, 1024);
      const uint64_t pd = noswz_desc(smem_u32(p_s), 128, 1024);
      const uint32_t d_s = tmem + TM_S, a_q = tmem + TM_Q, d_o = tmem + TM_O;
      int gi = 0, ui = 0;
      bool ok = true;
      auto v_stage = [&](int g) { return smem_u32(smem + OFF_V + g % kVStages * kVBlocks * K_CHUNK); };
      // P V of CTA tile g, the unit's first or a later one
      auto issue_pv = [&](int g, bool first) -> bool {
        if (!warp_wait(p_full, g & 1, p.err, abort_flag)) return false;
        tc_fence_after();
        const uint64_t vd = sw128_desc(v_stage(g), K_CHUNK, 1024);
        if (elect_one()) {
          if (first)
            umma_ss<0>(d_o, pd, vd, idesc_o);
          else
            umma_ss<1>(d_o, pd, vd, idesc_o);
          umma_ss<1>(d_o, pd + 16, vd + 128, idesc_o);
          umma_ss<1>(d_o, pd + 32, vd + 256, idesc_o);
          umma_ss<1>(d_o, pd + 48, vd + 384, idesc_o);
          mma_commit(pv_done);
          mma_commit(&v_empty[g % kVStages]);
        }
        __syncwarp();
        return true;
      };
      Unit x;
      for (; ok && take_unit(ui, x);) {
        const int ntiles = (x.hi - x.lo + kTile - 1) / kTile;
        if (!(ok = warp_wait(q_full, ui & 1, p.err, abort_flag))) break;
        ++ui;
        if (ntiles == 0) {
          if (elect_one()) mma_commit(q_empty);
          __syncwarp();
        }
        for (int j = 0; j < ntiles; ++j, ++gi) {
          if (!(ok = warp_wait(&k_full[gi & 1], (gi / 2) & 1, p.err, abort_flag))) break;
          if (gi >= 1 && !(ok = warp_wait(s_empty, (gi - 1) & 1, p.err, abort_flag))) break;
          tc_fence_after();
          const uint64_t xd = sw128_desc(smem_u32(smem + OFF_X), 16, 1024);
          const uint64_t yd = sw128_desc(smem_u32(smem + OFF_Y + gi % kYStages * kYBlocks * K_CHUNK), 16, 1024);
          const uint64_t vd = sw128_desc(v_stage(gi), 16, 1024);
          constexpr uint64_t kc = K_CHUNK >> 4, qc = Q_CHUNK >> 4;
          if (elect_one()) {
            // place c of the block order, 16 dims (32 bytes, 8 tensor-memory columns) per product; unrolled
            // (a loop over the blocks issues a third more slowly)
#pragma unroll
            for (int i = 0; i < 4 * kChunks; ++i) {
              const int c = i >> 2;
              const uint64_t bd = (c < kXBlocks ? xd + (uint64_t)c * kc : c < kXBlocks + kYBlocks ? yd + (uint64_t)(c - kXBlocks) * kc
                                                                       : vd + (uint64_t)(c - kXBlocks - kYBlocks) * kc) + (uint64_t)(i & 3) * 2;
              if (i == 0)
                umma_ss<0>(d_s, qd, bd, idesc_s);
              else if (c < kSmemQ)
                umma_ss<1>(d_s, qd + (uint64_t)c * qc + (uint64_t)(i & 3) * 2, bd, idesc_s);
              else
                umma_ts<1>(d_s, a_q + (uint32_t)((i - 4 * kSmemQ) * 8), bd, idesc_s);
              if (i == 4 * kXBlocks - 1) mma_commit(x_empty);
              if (i == 4 * (kXBlocks + kYBlocks) - 1) mma_commit(&y_empty[gi % kYStages]);
            }
            mma_commit(s_full);
            if (j == ntiles - 1) mma_commit(q_empty);
          }
          __syncwarp();
          if (j > 0 && !(ok = issue_pv(gi - 1, j == 1))) break;
        }
        if (ok && ntiles > 0) ok = issue_pv(gi - 1, ntiles == 1);
      }
      if (elect_one()) mma_commit(fin);
      __syncwarp();
      mbar_wait(fin, 0, p.err, nullptr);
    } else if (warp == R::kLookupWarp) {
      // ------------------------------------------------------------------ pool rows of the keys, tiles ahead
      int gi = 0;
      bool ok = true;
      int u = blockIdx.x;
      for (int k = 0; ok; ++k) {
        Unit x;
        x.rows = -1;
        for (; u < units;) {
          x = get_unit<kSrc>(p, u, lane == 0 && (u & 1) == 0 ? p.err : nullptr);
          if (x.rows > 0) break;
          u = next_unit(p, u);
          x.rows = -1;
        }
        if (k >= kUnitSlots && !(ok = warp_wait(&u_empty[k % kUnitSlots], ((k / kUnitSlots) - 1) & 1, p.err, abort_flag))) break;
        if (lane == 0) {
          unit_ring[k % kUnitSlots] = x;
          mbar_arrive(&u_full[k % kUnitSlots]);
        }
        if (x.rows < 0) break;
        u = next_unit(p, u);
        const int ntiles = (x.hi - x.lo + kTile - 1) / kTile;
        const bool report = x.v == 0;
        const int32_t* table = p.block_table + (int64_t)max(0, x.req) * p.max_blocks;
        if constexpr (!kQuant) {
          for (int j = 0; j < ntiles; ++j, ++gi) {
            const int lblk = x.lo / kTile + j;
            int page = lblk < p.max_blocks ? table[lblk] : -1;
            if (page < 0 || page >= p.num_blocks) {
              if (report) raise_error(p.err, DSA_DEVERR_BLOCK_ID);
              page = -1;
            }
            uint32_t may[2] = {~0u, ~0u};
            if (p.linear_pages && page >= 0) {
              page = x.req * p.linear_pages + lblk;
              const uint8_t* f = p.row_ok + (int64_t)page * kTile;
              may[0] = __ballot_sync(0xFFFFFFFFu, f[lane] != 0);
              may[1] = __ballot_sync(0xFFFFFFFFu, f[lane + 32] != 0);
            }
            if (gi >= kRowSlots && !(ok = warp_wait(&r_empty[gi % kRowSlots], ((gi / kRowSlots) - 1) & 1, p.err, abort_flag))) break;
            if (lane == 0) {
              row_ring[gi % kRowSlots * 4] = page;
              row_ring[gi % kRowSlots * 4 + 2] = (int32_t)may[0];
              row_ring[gi % kRowSlots * 4 + 3] = (int32_t)may[1];
              mbar_arrive(&r_full[gi % kRowSlots]);
            }
          }
          if (!ok) break;
          continue;
        }
        // lane: keys lane and lane + 32 of a tile; the selected positions are loaded a tile ahead
        auto position = [&](int j, int e) -> int {
          const int slot = x.lo + j * kTile + lane + 32 * e;
          if (slot >= x.hi) return -1;
          return kSrc == kSelected && p.idx ? p.idx[(int64_t)(x.row0 / p.H) * p.k + slot] : slot;
        };
        int ps[2] = {position(0, 0), position(0, 1)};
        for (int j = 0; j < ntiles; ++j, ++gi) {
          const int next[2] = {position(j + 1, 0), position(j + 1, 1)};
          int row[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            row[e] = -1;
            const bool seen = x.req >= 0 && ps[e] >= 0 && (kSrc != kSelected || ps[e] <= x.tok0);
            if (seen && ps[e] / kTile < p.max_blocks) row[e] = table[ps[e] / kTile];
            if (seen && (row[e] < 0 || row[e] >= p.num_blocks)) {
              if (report) raise_error(p.err, DSA_DEVERR_BLOCK_ID);
              row[e] = -1;
            }
            if (row[e] >= 0) row[e] = row[e] * kTile + ps[e] % kTile;
            if (kSrc == kSelected && !seen && ps[e] != -1 && x.req >= 0 && report) raise_error(p.err, DSA_DEVERR_INDEX);
          }
          if (gi >= kRowSlots && !(ok = warp_wait(&r_empty[gi % kRowSlots], ((gi / kRowSlots) - 1) & 1, p.err, abort_flag))) break;
          row_ring[gi % kRowSlots * kTile + lane] = row[0];
          row_ring[gi % kRowSlots * kTile + lane + 32] = row[1];
          __syncwarp();
          if (lane == 0) mbar_arrive(&r_full[gi % kRowSlots]);
          ps[0] = next[0];
          ps[1] = next[1];
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

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
    for (int e = 0; e < 16; ++e) a[e] = sp0 + e < n ? __ldg(src + (sp0 + e) * step) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
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
// a quantised key tile costs the attention ~4000 cycles, a bf16 one ~2500.  One warp per position of a request that
// has tokens; rows[(request, position)], rows of pages outside the pool are left out (never read).
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
    w[h] = __ldg(reinterpret_cast<const uint2*>(src + 256 * h) + lane);
    s[h] = __ldg(scale + row * 4 + 2 * h + (lane >> 4));
  }
  uint4 rope;
  if (lane < 8) rope = __ldg(reinterpret_cast<const uint4*>(src + kDv) + lane);
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
  // several requests: their units differ in size, and are handed out as CTAs become free
  p.next = nullptr;
  if (kSrc != kSelected && p.nsplit > 1 && p.num_reqs > 1) {
    p.next = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(p.part_lse) + up256((size_t)p.tiles * p.nsplit * p.prows * sizeof(float)));
    const cudaError_t e = cudaMemsetAsync(p.next, 0, sizeof(int), s);
    if (e != cudaSuccess) return e;
  }
  const int units = p.tiles * p.nsplit * 2;
  cudaError_t e = cudaSuccess;
  e = launch_pair<kSrc>(p, qmap, rmap, pmap, num_sms, s);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  cudaLaunchAttribute cattrs[2];
  const cudaLaunchConfig_t ccfg = launch_config(dim3(p.T, p.H), dim3(128), 0, s, cattrs);
  return cudaLaunchKernelEx(&ccfg, combine_kernel<kSrc != kSelected>, p);
}

// Row tiles of a batch of chunks (an upper bound: the device knows the chunks' sizes).
int64_t chunk_tiles(int num_tokens, int num_reqs, int H) { return first_tile(num_tokens, num_reqs, H); }

}  // namespace

// Key tiles of a split of a batch of chunks, at most.  Cost model in key-tile times: a unit costs its key
// tiles and a fixed ~4 (queries in, output out); units go round robin over the SMs, so on average half a unit is
// lost at the end; several splits cost the combine's launch and the partials' way to memory and back.  Only
// max_context and the numbers of tokens and requests are known here; of several requests the mean length is taken as
// 0.6 of the longest.
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
    const double units = 2.0 * tiles * (mean * n > 1.0 ? mean * n : 1.0);
    double cost = units <= num_sms ? per + 4.0 : (units / num_sms + 0.5) * (per + 4.0);
    if (n > 1) cost += 3.0 + 0.05 * tiles * n;
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
  // worth it from about three row tiles per request on (each key tile then saves at least six times ~1500 cycles for
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
  return launch<kSelected>(p, a, a.latent.data, a.latent.num_blocks, num_sms, s);
}

}  // namespace dsa
