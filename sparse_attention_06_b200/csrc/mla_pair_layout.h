// mla_pair_layout.h -- tile sizes of the MLA over 128 query rows (mla_pair.cu) and the map of a CTA's shared memory.
// Plain constants, so that a host program can check that what lives at the same time does not overlap.
#pragma once

namespace dsa {
namespace packed {

constexpr int kDqk = 576, kDv = 512, kHalf = 256;
constexpr int kRows = 128;               // query rows per tile (MMA M)
constexpr int kTile = 64;                // keys per tile = tokens per page
constexpr int kChunks = 9;               // 64-dim column blocks of a row
constexpr int kSmemQ = 3;                // Q blocks in shared memory (the first that Q K^T uses), the rest in tensor memory
constexpr int kFillWarps = 8, kKeysPerWarp = kTile / kFillWarps;
constexpr int kSoftmaxWarps = 4;         // 32 query rows each
constexpr int kUnitSlots = 2, kUnitBytes = 40;

// A tile's blocks in the order Q K^T uses them: X0 (RoPE), X1, Y0, Y1, Y2 (the values of the other
// half), V0 .. V3 (this half's values).
constexpr int kXBlocks = 2, kYBlocks = 3, kVBlocks = 4;

constexpr int K_CHUNK = kTile * 128;
constexpr int Q_CHUNK = kRows * 128;
constexpr int P_BYTES = kRows * kTile * 2;
constexpr int V_BYTES = kVBlocks * K_CHUNK;
constexpr int OFF_Q = 0;
constexpr int OFF_P = OFF_Q + kSmemQ * Q_CHUNK;            // [2]: of the page of CTA 0, of CTA 1
constexpr int OFF_Y = OFF_P + 2 * P_BYTES;
constexpr int OFF_X = OFF_Y + kYBlocks * K_CHUNK;
constexpr int OFF_V = OFF_X + kXBlocks * K_CHUNK;          // [2] own page, [1] the other
constexpr int OFF_BAR = OFF_V + 3 * V_BYTES;
constexpr int NBAR = 48;
constexpr int kSlots = 4;
constexpr int OFF_MASK = OFF_BAR + NBAR * 8;               // [slot] keys of the own page with a row to see, a byte per fill warp
constexpr int OFF_POISON = OFF_MASK + kSlots * 8;          // [slot] rows with NaN or infinity
constexpr int OFF_STATS = OFF_POISON + kSlots * 8;         // 1 / l of each row (last unit)
constexpr int OFF_MAX = OFF_STATS + kRows * 4;             // [2][128] values of the other CTA's rows
constexpr int OFF_UNIT = OFF_MAX + 2 * kRows * 4;          // [2] units in hand
constexpr int OFF_ROWS = OFF_UNIT + kUnitSlots * kUnitBytes;  // [slot] bf16: own page, other page, masks of their rows that may be
                                                           // read; quantised: [2][64] pool row of each key of either, -1: none
constexpr int OFF_MAIL = OFF_ROWS + kSlots * 2 * kTile * 4;           // [4] units from CTA 0
constexpr int OFF_MISC = OFF_MAIL + 16;
constexpr int SMEM = OFF_MISC + 16;
static_assert(SMEM <= 232448, "shared memory budget");
static_assert(OFF_ROWS % 16 == 0 && OFF_MASK % 8 == 0, "alignment");

// A softmax warp's 32 rows of P, in CTA v of the pair, and where it stages its outputs.  One softmax warp may be a unit
// ahead of another (no barrier stands between a warp's epilogue and the others' first P of the next unit), so an output
// is staged where no other warp writes: in the warp's own rows of P.
constexpr int kWarpPBytes = P_BYTES / kSoftmaxWarps, kStageBytes = 2048;
constexpr int p_offset(int v, int warp) { return OFF_P + v * P_BYTES + warp * kWarpPBytes; }
constexpr int stage_offset(int v, int warp) { return p_offset(v, warp); }
static_assert(kStageBytes <= kWarpPBytes, "an output is staged within the warp's own P");

}  // namespace packed
}  // namespace dsa
