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
hipError_t attn_bwd_narrow_launch_1_96(const AttnParams&, hipStream_t);
hipError_t attn_bwd_narrow_launch_1_128(const AttnParams&, hipStream_t);

hipError_t attn_combine_launch(const AttnParams&, bool bf16, hipStream_t);
hipError_t attn_stats_launch(const AttnParams&, bool bf16, hipStream_t);

// The forward kernels' tile shapes, by rule on type, head size and rows.
// Waves of a workgroup with rows of their own: 0 selects the kernel whose waves
// own keys (up to 32 rows, one or two column groups).
constexpr int fwd_columns(bool bf16) { return bf16 ? 2 : 1; }
constexpr int fwd_key_tile(bool bf16, int dp) { return bf16 && dp <= 160 ? 64 : 32; }
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
// Above a head size of 160 they spill to memory in the loop over the keys (bf16 at 192,
// 224, 256: 12, 69, 66 registers; fp32: 28, 90, 114).  One row, 41880 keys, 16 heads, no
// mask, eight waves and four, us: bf16 at 96 57 and 53, 128 77 and 78, 160 91 and 89, 192
// 116 and 106, 224 220 and 119, 256 179 and 130; fp32 at 64 72 and 83, 128 134 and 135,
// 160 164 and 166, 192 267 and 191, 224 566 and 226, 256 311 and 255.  32 x 5 rows, 1000
// keys, 8 heads of 64: bf16 14.2 and 13.8 with a mask, fp32 23.8 and 25.6.
constexpr int step_key_tile(bool bf16) { return bf16 ? 32 : 16; }
constexpr int step_max_waves(int dp) { return dp <= 160 ? 8 : 4; }
constexpr int step_waves(bool bf16, int dp, int rows, int S) {
  return step_columns(bf16, dp, rows) == 1 && S > 4 * step_key_tile(bf16) ? step_max_waves(dp) : 4;
}
// keys that a workgroup takes together
constexpr int fwd_keys_per_block(bool bf16, int dp, int rows, int S) {
  return rows <= 32 ? step_waves(bf16, dp, rows, S) * step_key_tile(bf16) : fwd_key_tile(bf16, dp);
}
// 16-column groups of a backward wave: two where operands and sums of that many fit the registers
constexpr int bwd_columns(bool bf16, int dp) { return bf16 && dp <= 128 ? 2 : 1; }
// registers that these take on the key side
constexpr int bwd_registers(bool bf16, int dp) { return bwd_columns(bf16, dp) * dp * (bf16 ? 12 : 16) / 16; }
// bf16 keeps two waves a SIMD: where a wave's registers are short (192 of 256
// here), v's operands lie in LDS, in workgroups of eight waves; elsewhere four
// waves, whose barriers hold up fewer (D 80, 32 x 200 rows over 777 keys: 78 us, 86
// with eight).
constexpr bool bwd_short(bool bf16, int dp) { return bf16 && bwd_registers(bf16, dp) >= 192; }
constexpr int bwd_waves(bool bf16, int dp) { return bwd_short(bf16, dp) ? 8 : 4; }
constexpr int bwd_waves_per_simd(bool bf16, int dp) { return bf16 || bwd_registers(bf16, dp) < 192 ? 2 : 1; }
// One group where there are few rows and keys: more, smaller workgroups then hide
// each other's latency (300 rows, 400 keys at most, 192 heads of 64: 47 us, 55 with
// two; 40 and 50, 256 heads of 128: 13 and 19; 200 and 777, 128 heads of 80: 78 and
// 72; 1000 and 1000, 64 heads of 64: 99 and 86).
constexpr bool bwd_narrow(bool bf16, int dp, int rows, int S) {
  return bwd_columns(bf16, dp) == 2 && rows <= 512 && S <= 512;
}
constexpr int bwd_narrow_waves_per_simd(int dp) { return dp <= 64 ? 4 : 3; }
constexpr int bwd_row_tile(bool bf16, int dp) { return bf16 && dp <= 64 ? 64 : 32; }
constexpr int bwd_key_tile(bool bf16, int dp) { return bf16 && dp <= 160 ? 64 : 32; }

}  // namespace lstm
