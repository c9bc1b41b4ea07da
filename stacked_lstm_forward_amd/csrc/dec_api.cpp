// C-ABI entry points of the decoder's attention (host side): argument checks,
// the split of the key axis, workspace layout, launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "dec_attn_launch.h"
#include "decoder/lstm_dec.h"  // include/ is on the include path

using namespace lstm;

namespace {

typedef hipError_t (*AttnLaunch)(const AttnParams&, hipStream_t);

#define DEC_ROW(kind, bf)                                                                                    \
  {attn_##kind##_launch_##bf##_32,  attn_##kind##_launch_##bf##_64,  attn_##kind##_launch_##bf##_96,         \
   attn_##kind##_launch_##bf##_128, attn_##kind##_launch_##bf##_160, attn_##kind##_launch_##bf##_192,        \
   attn_##kind##_launch_##bf##_224, attn_##kind##_launch_##bf##_256}
const AttnLaunch kFwd[2][8] = {DEC_ROW(fwd, 0), DEC_ROW(fwd, 1)};
const AttnLaunch kBwd[2][8] = {DEC_ROW(bwd, 0), DEC_ROW(bwd, 1)};
#undef DEC_ROW
const AttnLaunch kBwdNarrow[2] = {attn_bwd_narrow_launch_1_32, attn_bwd_narrow_launch_1_64};

// Lengths and row counts are held in 32 bits, and the kernels' counters step past
// them by less than 4096 (two tiles of all waves).
constexpr long long kMaxCount = (1ll << 31) - 4096;
constexpr int kComputeUnits = 256;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Strides are multiples of 16 bytes; outputs' elements must not coincide, which
// is left to the caller like any other overlap.
bool stride_ok(const lstm_attn_stride_t& s, int size) {
  const int64_t unit = 16 / size;
  return s.b % unit == 0 && s.t % unit == 0 && s.h % unit == 0;
}

lstm_status_t check_desc(const lstm_attn_desc_t* d, bool train) {
  if (!d) return LSTM_ERR_INVALID_ARG;
  if (d->B < 1 || d->Tq < 1 || d->S < 0 || d->Hq < 1 || d->Hkv < 1 || d->D < 1) return LSTM_ERR_INVALID_ARG;
  if (d->dtype != LSTM_F32 && d->dtype != LSTM_BF16) return LSTM_ERR_INVALID_ARG;
  if (d->Hq % d->Hkv != 0) return LSTM_ERR_INVALID_ARG;
  if (!(d->scale >= 0.f) || std::isinf(d->scale * kLog2e)) return LSTM_ERR_INVALID_ARG;  // the kernels' factor
  const int size = d->dtype == LSTM_BF16 ? 2 : 4;
  if (!stride_ok(d->q, size) || !stride_ok(d->k, size) || !stride_ok(d->v, size) || !stride_ok(d->o, size))
    return LSTM_ERR_UNSUPPORTED;
  if (train && (!stride_ok(d->dout, size) || !stride_ok(d->dq, size) || !stride_ok(d->dk, size) ||
                !stride_ok(d->dv, size)))
    return LSTM_ERR_UNSUPPORTED;
  if (d->D % 8 != 0 || d->D > 256) return LSTM_ERR_UNSUPPORTED;
  if ((long long)d->B * d->Hq > kMaxCount || (long long)d->B * d->Hq * d->Tq > kMaxCount ||
      (long long)d->B * d->S > kMaxCount)
    return LSTM_ERR_UNSUPPORTED;
  // the backward's workgroups, of 64 rows or keys at least (the forward's are no more than its rows)
  const long long rows = (long long)d->Tq * (d->Hq / d->Hkv), tiles = (rows + 63) / 64 + ((long long)d->S + 63) / 64;
  if (train && (long long)d->B * d->Hkv > kMaxCount / tiles) return LSTM_ERR_UNSUPPORTED;
  return LSTM_OK;
}

AttnStride bytes(const lstm_attn_stride_t& s, int size) { return AttnStride{s.b * size, s.t * size, s.h * size}; }

AttnParams params(const lstm_attn_desc_t* d) {
  AttnParams p = {};
  const int size = d->dtype == LSTM_BF16 ? 2 : 4;
  p.B = d->B, p.Tq = d->Tq, p.S = d->S, p.Hq = d->Hq, p.Hkv = d->Hkv, p.G = d->Hq / d->Hkv, p.D = d->D;
  p.rows = p.Tq * p.G;
  p.scale = d->scale != 0.f ? d->scale : 1.f / std::sqrt((float)d->D);
  p.scale_log2 = p.scale * kLog2e;
  p.sq = bytes(d->q, size), p.sk = bytes(d->k, size), p.sv = bytes(d->v, size), p.so = bytes(d->o, size);
  p.sdo = bytes(d->dout, size), p.sdq = bytes(d->dq, size), p.sdk = bytes(d->dk, size), p.sdv = bytes(d->dv, size);
  p.o_rest = size == 2 ? (char*)d->o_rest : nullptr;
  p.nsplit = 1;
  p.kv_per_split = p.S;
  return p;
}

// Splits the key axis where the row tiles alone leave compute units idle: one
// workgroup a compute unit, none with less than four key tiles (two of the tiles
// that the waves of a few-rows workgroup take together).
void plan_fwd(const lstm_attn_desc_t* d, AttnParams* p) {
  const bool bf = d->dtype == LSTM_BF16;
  const int dp = (d->D + 31) / 32 * 32;
  const int per = fwd_rows_per_block(bf, dp, p->rows), kt = fwd_keys_per_block(bf, dp, p->rows, p->S);
  p->tiles = (p->rows + per - 1) / per;
  const long long blocks = (long long)p->B * p->Hkv * p->tiles;
  const int ktiles = (p->S + kt - 1) / kt;
  long long n = (kComputeUnits + blocks - 1) / blocks;
  const int least = p->rows <= 32 ? 2 : 4;
  if (n > ktiles / least) n = ktiles / least;
  if (n < 1) n = 1;
  const int each = (int)((ktiles + n - 1) / n);
  p->nsplit = each > 0 ? (ktiles + each - 1) / each : 1;
  p->kv_per_split = p->nsplit > 1 ? each * kt : p->S;
  p->blocks = (int)(blocks * p->nsplit);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t fwd_parts(const AttnParams& p, size_t* ml_at) {
  if (p.nsplit == 1) return *ml_at = 0;
  const size_t n = (size_t)p.B * p.Hkv * p.rows * p.nsplit;
  *ml_at = round256(n * p.D * sizeof(float));
  return *ml_at + round256(n * 2 * sizeof(float));
}

bool ws_ok(const void* ws) { return ws && (reinterpret_cast<uintptr_t>(ws) & 255) == 0; }

int dp_index(int D) { return (D + 31) / 32 - 1; }

}  // namespace

extern "C" {

lstm_status_t lstm_attn_validate(const lstm_attn_desc_t* d, int train) { return check_desc(d, train != 0); }

size_t lstm_attn_workspace_size(const lstm_attn_desc_t* d) {
  if (check_desc(d, false) != LSTM_OK) return 0;
  AttnParams p = params(d);
  plan_fwd(d, &p);
  size_t at;
  const size_t n = fwd_parts(p, &at);
  return n ? n : 256;
}

size_t lstm_attn_bwd_workspace_size(const lstm_attn_desc_t* d) {
  if (check_desc(d, true) != LSTM_OK) return 0;
  return round256((size_t)d->B * d->Hq * d->Tq * 2 * sizeof(float));
}

lstm_status_t lstm_attn_fwd(const lstm_attn_desc_t* d, const void* q, const void* k, const void* v,
                            const int32_t* kv_len, const uint8_t* key_mask, void* o, float* lse, void* ws,
                            hipStream_t stream) {
  const lstm_status_t st = check_desc(d, false);
  if (st != LSTM_OK) return st;
  if (!q || !o || (d->S > 0 && (!k || !v))) return LSTM_ERR_INVALID_ARG;
  if (!aligned4(kv_len) || !aligned4(lse)) return LSTM_ERR_INVALID_ARG;
  if (!aligned16(d->o_rest)) return LSTM_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return LSTM_ERR_UNSUPPORTED;
  if (!ws_ok(ws)) return LSTM_ERR_WORKSPACE;
  AttnParams p = params(d);
  plan_fwd(d, &p);
  p.q = (const char*)q, p.k = (const char*)k, p.v = (const char*)v, p.o = (char*)o, p.lse = lse;
  p.kv_len = kv_len, p.key_mask = key_mask;
  size_t at;
  fwd_parts(p, &at);
  p.part_o = (float*)ws;
  p.part_ml = (float*)((char*)ws + at);
  const bool bf = d->dtype == LSTM_BF16;
  if (kFwd[bf][dp_index(d->D)](p, stream) != hipSuccess) return LSTM_ERR_HIP;
  if (p.nsplit > 1 && attn_combine_launch(p, bf, stream) != hipSuccess) return LSTM_ERR_HIP;
  return LSTM_OK;
}

lstm_status_t lstm_attn_bwd(const lstm_attn_desc_t* d, const void* q, const void* k, const void* v,
                            const int32_t* kv_len, const uint8_t* key_mask, const void* o, const float* lse,
                            const void* dout, void* dq, void* dk, void* dv, void* ws, hipStream_t stream) {
  const lstm_status_t st = check_desc(d, true);
  if (st != LSTM_OK) return st;
  if (!q || !o || !lse || !dout || !dq || (d->S > 0 && (!k || !v || !dk || !dv))) return LSTM_ERR_INVALID_ARG;
  if (!aligned4(kv_len) || !aligned4(lse)) return LSTM_ERR_INVALID_ARG;
  for (const void* x : {q, k, v, o, dout, (const void*)dq, (const void*)dk, (const void*)dv, (const void*)d->o_rest})
    if (!aligned16(x)) return LSTM_ERR_UNSUPPORTED;
  if (!ws_ok(ws)) return LSTM_ERR_WORKSPACE;
  AttnParams p = params(d);
  p.q = (const char*)q, p.k = (const char*)k, p.v = (const char*)v, p.o_in = (const char*)o, p.lse_in = lse;
  p.dout = (const char*)dout, p.dq = (char*)dq, p.dk = (char*)dk, p.dv = (char*)dv;
  p.kv_len = kv_len, p.key_mask = key_mask;
  p.stats = (float*)ws;
  const bool bf = d->dtype == LSTM_BF16;
  if (attn_stats_launch(p, bf, stream) != hipSuccess) return LSTM_ERR_HIP;
  const int at = dp_index(d->D);
  const AttnLaunch run = bwd_narrow(bf, (at + 1) * 32, p.rows, p.S) ? kBwdNarrow[at] : kBwd[bf][at];
  if (run(p, stream) != hipSuccess) return LSTM_ERR_HIP;
  return LSTM_OK;
}

}  // extern "C"
