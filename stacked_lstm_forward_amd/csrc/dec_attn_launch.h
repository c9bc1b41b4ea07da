// Launchers of the attention kernels, one per element type (0 fp32, 1 bf16) and
// padded head size.
#pragma once

#include "dec_attn.h"

namespace lstm {

#define DEC_ATTN_DECLARE(dp)                                                     \
  hipError_t attn_fwd_launch_0_##dp(const AttnParams&, hipStream_t);             \
  hipError_t attn_fwd_launch_1_##dp(const AttnParams&, hipStream_t);             \
  hipError_t attn_bwd_launch_0_##dp(const AttnParams&, hipStream_t);             \
  hipError_t attn_bwd_launch_1_##dp(const AttnParams&, hipStream_t);
DEC_ATTN_DECLARE(32)
DEC_ATTN_DECLARE(64)
DEC_ATTN_DECLARE(96)
DEC_ATTN_DECLARE(128)
DEC_ATTN_DECLARE(160)
DEC_ATTN_DECLARE(192)
DEC_ATTN_DECLARE(224)
DEC_ATTN_DECLARE(256)
#undef DEC_ATTN_DECLARE
hipError_t attn_bwd_narrow_launch_1_32(const AttnParams&, hipStream_t);
hipError_t attn_bwd_narrow_launch_1_64(const AttnParams&, hipStream_t);

hipError_t attn_combine_launch(const AttnParams&, bool bf16, hipStream_t);
hipError_t attn_stats_launch(const AttnParams&, bool bf16, hipStream_t);

// The forward kernels' tile shapes, by rule on type, head size and rows.
// Waves of a workgroup with rows of their own: 0 selects the kernel whose waves
// own keys (up to 32 rows, one or two column groups).
constexpr int fwd_columns(bool bf16) { return bf16 ? 2 : 1; }
// (fp32 above 192: with tiles of 32 a wave of eight spills beside a tile's own sums; 32
// heads of 1000 rows and keys at 224 and 256 263 and 290 us, with four waves 287 and 342,
// spilling 323 and 376)
constexpr int fwd_key_tile(bool bf16, int dp) { return bf16 ? (dp <= 160 ? 64 : 32) : dp > 192 ? 16 : 32; }
// eight waves share a tile where their operands and sums fit 256 registers a lane
constexpr int fwd_max_waves(bool bf16, int dp) { return bf16 && dp > 128 ? 4 : 8; }
constexpr int fwd_waves(bool bf16, int dp, int rows) {
  return rows <= 32 ? 0 : rows <= 64 * fwd_columns(bf16) ? 4 : fwd_max_waves(bf16, dp);
}
// column groups of the few-rows kernel: two where they fit the registers
constexpr int step_max_columns(bool bf16, int dp) { return dp <= (bf16 ? 192 : 128) ? 2 : 1; }
constexpr int step_columns(bool bf16, int dp, int rows) { return rows <= 16 ? 1 : step_max_columns(bf16, dp); }
constexpr int fwd_rows_per_block(bool bf16, int dp, int rows) {
  return rows <= 32 ? 16 * step_columns(bf16, dp, rows) : fwd_waves(bf16, dp, rows) * 16 * fwd_columns(bf16);
}
// Waves of the few-rows kernel: eight where four would not take all keys at once and
// a wave's operands, sums and loads ahead fit the 256 registers that eight leave it.
// Above a head size of 160 (fp32 128) they spill to memory in the loop over the keys.
// One row, 41880 keys, 16 heads, no mask, eight waves and four, us: bf16 at 96 57 and 53,
// 128 77 and 78, 160 91 and 89, 192 116 and 106, 224 220 and 119, 256 179 and 130; fp32 at
// 64 72 and 83, 128 134 and 135, 160 168 and 165, 192 267 and 191, 224 566 and 226, 256 311
// and 255.  32 x 5 rows, 1000 keys, 8 heads: bf16 at 64 14.2 and 13.8 with a mask; fp32 at
// 64 23.8 and 25.6, at 160 66 and 61.
constexpr int step_key_tile(bool bf16) { return bf16 ? 32 : 16; }
constexpr int step_max_waves(bool bf16, int dp) { return dp <= (bf16 ? 160 : 128) ? 8 : 4; }
constexpr int step_waves(bool bf16, int dp, int rows, int S) {
  return step_columns(bf16, dp, rows) == 1 && S > 4 * step_key_tile(bf16) ? step_max_waves(bf16, dp) : 4;
}
// keys that a workgroup takes together
constexpr int fwd_keys_per_block(bool bf16, int dp, int rows, int S) {
  return rows <= 32 ? step_waves(bf16, dp, rows, S) * step_key_tile(bf16) : fwd_key_tile(bf16, dp);
}
// 16-column groups of a backward wave, bf16: two for heads of 64 at most; beyond that
// their operands, sums and two-part products spill 32 registers and more.  us with one
// and with two groups, 48 heads (sentences' heads) of 2048 rows and up to 3001 keys: 286
// and 257 at 24, 372 and 335 at 64, 424 both at 96, 549 and 583 at 128; 128 heads of 100
// rows and 3000 keys: 94 and 76, 91 and 84, 131 and 154, 172 and 225; 3000 rows and 100
// keys: 118 and 122, 145 and 146, 223 and 257, 264 and 250.
constexpr int bwd_columns(bool bf16, int dp) { return bf16 && dp <= 64 ? 2 : 1; }
// For these, one group too where there are few rows and keys: more, smaller workgroups
// then hide each other's latency.  us with one and with two groups, heads of 64: 768 of
// 120 rows and 130 keys 45 and 61, 192 of 300 and 400 48 and 59; 128 of 600 and 600 73
// and 75 (heads of 32: 58 both), 64 of 1000 and 1000 90 and 94 (69 and 65).
constexpr bool bwd_narrow(bool bf16, int dp, int rows, int S) {
  return bwd_columns(bf16, dp) == 2 && rows <= 512 && S <= 512;
}
constexpr int kBwdNarrowWavesPerSimd = 4;
// registers that operands and sums take on the key side
constexpr int bwd_registers(bool bf16, int dp) { return bwd_columns(bf16, dp) * dp * (bf16 ? 12 : 16) / 16; }
// bf16 runs two waves a SIMD at least (three at 96 and 128).  At 256, where the operands
// and sums of a wave take 192 of the 256 registers that this leaves it, v's operands lie
// in LDS, in workgroups of eight waves.  At 224 the loop spills 27 registers; with v's
// operands in LDS it does not, which is faster for long rows and slower for short ones
// (32 heads of 1000 rows and keys: 179 us, now 199; 256 heads of 120 and 130: 77, now 65).
constexpr bool bwd_short(bool bf16, int dp) { return bf16 && bwd_registers(bf16, dp) >= 192; }
constexpr int bwd_waves(bool bf16, int dp) { return bwd_short(bf16, dp) ? 8 : 4; }
// fp32 runs three up to 64 (512 heads of 100 rows and 120 keys: 73 us, 80 with two), two
// up to 128, then one.
constexpr int bwd_waves_per_simd(bool bf16, int dp) {
  return bf16 ? (dp > 64 && dp <= 128 ? 3 : 2) : dp <= 64 ? 3 : bwd_registers(bf16, dp) < 192 ? 2 : 1;
}
// Tiles of 64 where they leave LDS to the workgroups that the registers allow (at 160
// with key tiles of 64 one workgroup of four waves fits: 269 us, now 147, for 32 heads
// of 1000 rows and keys).
constexpr int bwd_row_tile(bool bf16, int dp) { return bf16 && dp <= 64 ? 64 : 32; }
constexpr int bwd_key_tile(bool bf16, int dp) { return bf16 && dp <= 64 ? 64 : 32; }

}  // namespace lstm
