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

hipError_t attn_combine_launch(const AttnParams&, bool bf16, hipStream_t);
hipError_t attn_delta_launch(const AttnParams&, bool bf16, hipStream_t);

// Rows a forward workgroup owns, keys a backward workgroup owns and rows its
// query-side part owns (the kernels' tile shapes).
constexpr int fwd_rows_per_block(bool bf16) { return bf16 ? 128 : 64; }
constexpr int fwd_key_tile(bool bf16) { return bf16 ? 64 : 32; }
// 16-column groups of a backward wave: two where operands and sums of that many fit the registers
constexpr int bwd_columns(bool bf16, int dp) { return bf16 && dp <= 128 ? 2 : 1; }

}  // namespace lstm
