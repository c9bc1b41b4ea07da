// Attention over encoder outputs, forward.  One translation unit per element
// type and padded head size (DEC_BF16, DEC_DP).
#include "dec_attn.h"
#include "dec_attn_launch.h"

namespace lstm {
namespace {

#if DEC_BF16
typedef uint16_t ET;
#else
typedef float ET;
#endif
constexpr int DP = DEC_DP;

// The maximum of a tile's scores (base-2 units), one per column.
template <int QC, int KT>
__device__ __forceinline__ void tile_max(const f32x4 (&x)[KT / 16][QC], float (&mn)[QC], float scale_log2) {
#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    float mx = x[0][qc][0];
#pragma unroll
    for (int kt = 0; kt < KT / 16; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, x[kt][qc][i]);
    mn[qc] = col_max(mx) * scale_log2;
  }
}

// The maximum in use stays until it is 2^8 behind: exponentials up to 2^8 are as
// exact as those below 1, and o is rescaled for few tiles only.
template <int QC, int NTILES>
__device__ __forceinline__ void raise_max(const float (&mn)[QC], f32x4 (&o)[NTILES][QC], float (&m)[QC],
                                          float (&l)[QC]) {
#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    if (__any(mn[qc] > m[qc] + 8.f)) {
      const float mu = fmaxf(m[qc], mn[qc]);
      const float alpha = mu == -INFINITY ? 1.f : exp2_fast(m[qc] - mu);
      m[qc] = mu;
      l[qc] *= alpha;
#pragma unroll
      for (int n = 0; n < NTILES; ++n) o[n][qc] *= alpha;
    }
  }
}

// Scores become exponentials, their sum goes to l (a tile's by itself first: a long
// sum then takes one rounding of its own size a tile, not one a key).
template <int QC, int KT>
__device__ __forceinline__ void tile_exp(f32x4 (&x)[KT / 16][QC], const float (&m)[QC], float (&l)[QC],
                                         float scale_log2) {
#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    const float mu = m[qc] == -INFINITY ? 0.f : m[qc];
    float sum = 0.f;
#pragma unroll
    for (int kt = 0; kt < KT / 16; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = exp2_fast(fmaf(x[kt][qc][i], scale_log2, -mu));
        x[kt][qc][i] = e;
        sum += e;
      }
    l[qc] += sum;
  }
}

template <typename T, int DP, int QC, int KT, int NTILES>
__device__ __forceinline__ void softmax_tile(f32x4 (&x)[KT / 16][QC], f32x4 (&o)[NTILES][QC], float (&m)[QC],
                                             float (&l)[QC], float scale_log2) {
  float mn[QC];
  tile_max<QC, KT>(x, mn, scale_log2);
  raise_max<QC, NTILES>(mn, o, m, l);
  tile_exp<QC, KT>(x, m, l, scale_log2);
}

// One column group's results, to o and lse or to the parts of a split.
template <typename T, int DP, int QC, int NTILES>
__device__ __forceinline__ void store_rows(const AttnParams& p, int b, int hk, int bh, int split, int row0, int qc,
                                           const f32x4 (&o)[NTILES][QC], float m, float l, int lane) {
  const int r = row0 + qc * 16 + (lane & 15);
  if (r >= p.rows) return;
  if (p.nsplit > 1) {
    const long long at = ((long long)bh * p.rows + r) * p.nsplit + split;
    store_cols_f32<T, DP, NTILES, QC>(p.part_o + at * p.D, o, qc, p.D, lane);
    if (lane < 16) {
      p.part_ml[at * 2] = m;
      p.part_ml[at * 2 + 1] = l;
    }
    return;
  }
  const int t = r / p.G, hq = hk * p.G + r % p.G;
  char* rest = p.o_rest ? p.o_rest + ((long long)bh * p.rows + r) * p.D * 2 : nullptr;
  store_cols<T, DP, NTILES, QC>(p.o + b * p.so.b + t * p.so.t + hq * p.so.h, o, qc, l == 0.f ? 0.f : 1.f / l, p.D,
                                lane, rest);
  if (lane < 16 && p.lse)
    p.lse[((long long)b * p.Hq + hq) * p.Tq + t] = (m == -INFINITY ? 0.f : m) * kLn2 + logf(l);
}

// Each wave owns 16*QC rows (columns of S^T), the workgroup's NW waves share
// the KT keys of a tile in LDS, so that a byte read from there feeds QC products.
// One pass over the keys with the running maximum and sum.  Long rows are bound by
// matrix and vector work that two waves a SIMD overlap only partly (matrix pipe busy
// 45 % of the time, vector pipe 48 %, no bank conflicts): 8 x 2048 rows, 4096 keys, 32
// heads of 128, bf16 1.52 ms = 722 TFLOP/s (1084 with the second product of p), where a
// library product of 8192^3 reaches 1108.  With p rounded once it took 1.21 ms, and
// then one tile at a time instead of two interleaved 1.57.  Short ones (64 x 200 rows,
// 331 keys, 4 heads of 64: 19.5 us, 5.9 for its bytes) are bound by the latency of six
// dependent tiles, whose loads are issued one tile ahead.  Heads of 136 to 256 in bf16
// run four waves of up to 476 registers, one a SIMD: every tile's latency shows (4 x
// 2000 rows, 2000 keys, 8 heads of 256: 287 us, 118 for its products).
template <typename T, int DP, int QC, int NW, int KT>
__global__ void __launch_bounds__(NW * 64) attn_fwd_kernel(AttnParams p) {
  constexpr int SZ = AT<T>::SZ, NT = NW * 64, PB = Pitch<T, DP>::B;
  constexpr int NCH = DP * SZ / 64;  // 64-byte chunks of a row
  constexpr int NTILES = DP / 16;
  // two buffers: a tile is written while its predecessor is read, one barrier a tile
  __shared__ __align__(16) char skb[2][KT * PB];
  __shared__ __align__(16) char svb[2][KT * PB];
  __shared__ __align__(16) float sbiasb[2][KT];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const unsigned block = grid_block();
  if (block >= (unsigned)p.blocks) return;
  const int item = xcd_item(block, p.blocks);
  const int tile = item % p.tiles, rest = item / p.tiles;
  const int split = rest % p.nsplit, pair = rest / p.nsplit;
  const int b = pair % p.B, hk = pair / p.B, bh = b * p.Hkv + hk;
  const int db = p.D * SZ;

  const int s0 = split * p.kv_per_split;
  const int s1 = s0 + min(keys_of(p, b) - s0, p.kv_per_split);
  const char* kb = p.k + b * p.sk.b + hk * p.sk.h;
  const char* vb = p.v + b * p.sv.b + hk * p.sv.h;
  const uint8_t* mb = p.key_mask ? p.key_mask + (long long)b * p.S : nullptr;

  // query fragments
  const int row0 = (tile * NW + wave) * 16 * QC;
  uint4 qf[QC][NCH];
#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    const int r = row0 + qc * 16 + (lane & 15);
    const bool ok = r < p.rows;
    const int t = ok ? r / p.G : 0, gh = ok ? r % p.G : 0;
    const char* qr = p.q + b * p.sq.b + t * p.sq.t + (hk * p.G + gh) * p.sq.h;
#pragma unroll
    for (int c = 0; c < NCH; ++c) qf[qc][c] = load16(qr, c * 64 + (lane >> 4) * 16, db, ok);
  }

  f32x4 o[NTILES][QC];
  float m[QC], l[QC];
#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    m[qc] = -INFINITY;
    l[qc] = 0.f;
#pragma unroll
    for (int n = 0; n < NTILES; ++n) o[n][qc] = (f32x4){0.f, 0.f, 0.f, 0.f};
  }

  TileCopy<T, DP, KT, NT> ck, cv;
  uint8_t rb = 0;
  auto load_k = [&](int s) {
    ck.load(s, s1, mb, tid, db);
    if (tid < KT) rb = s + tid < s1 ? (mb ? mb[s + tid] : 1) : 0;
  };
  auto store_k = [&](int buf, int s) {
    ck.store(skb[buf], s, s1, mb, tid, db, ck.m);
    if (tid < KT) sbiasb[buf][tid] = rb ? 0.f : -INFINITY;
  };
  // -inf where a tile has keys left out (whatever q holds: a row without keys gives 0)
  auto leave_out = [&](f32x4 (&x)[KT / 16][QC], int s, int buf) {
    if (mb || s + KT > s1) {
#pragma unroll
      for (int kt = 0; kt < KT / 16; ++kt) {
        const f32x4 bias = *reinterpret_cast<const f32x4*>(sbiasb[buf] + kt * 16 + (lane >> 4) * 4);
#pragma unroll
        for (int qc = 0; qc < QC; ++qc)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[kt][qc][i] = bias[i] == 0.f ? x[kt][qc][i] : -INFINITY;
      }
    }
  };

  // Tile i's exponentials are taken beside the matrix products of tile i+1's scores.
  // k is a tile ahead of v in LDS; a buffer is written one barrier after its last read.
  f32x4 xa[KT / 16][QC], xb[KT / 16][QC];
  float mn[QC];
  if (s0 < s1) {
    ck.init(kb, p.sk.t, s0, tid, db);
    cv.init(vb, p.sv.t, s0, tid, db);
    load_k(s0);
    cv.load(s0, s1, mb, tid, db);
    store_k(0, s0);
    if (s0 + KT < s1) load_k(s0 + KT);
    cv.store(svb[0], s0, s1, mb, tid, db, cv.m);
    if (s0 + KT < s1) store_k(1, s0 + KT);
    __syncthreads();
    mma_rows0<T, DP, QC, KT>(xa, skb[0], qf, lane);
    leave_out(xa, s0, 0);
    tile_max<QC, KT>(xa, mn, p.scale_log2);
    __syncthreads();
  }
  auto step = [&](f32x4 (&x)[KT / 16][QC], f32x4 (&y)[KT / 16][QC], int s, int buf) {
    const bool more = s + KT < s1, more2 = s + 2 * KT < s1;
    if (more2) load_k(s + 2 * KT);
    if (more) cv.load(s + KT, s1, mb, tid, db);
    raise_max<QC, NTILES>(mn, o, m, l);
    mma_rows0<T, DP, QC, KT>(y, skb[buf ^ 1], qf, lane);  // of stale rows after the last tile: not used
    tile_exp<QC, KT>(x, m, l, p.scale_log2);
    mma_tr<T, DP, QC, KT, NTILES>(o, svb[buf], x, lane);
    leave_out(y, s + KT, buf ^ 1);
    tile_max<QC, KT>(y, mn, p.scale_log2);
    if (more2) store_k(buf, s + 2 * KT);
    if (more) cv.store(svb[buf ^ 1], s + KT, s1, mb, tid, db, cv.m);
    __syncthreads();
  };
  for (int s = s0; s < s1; s += 2 * KT) {
    step(xa, xb, s, 0);
    if (s + KT >= s1) break;
    step(xb, xa, s + KT, 1);
  }

#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    store_rows<T, DP, QC, NTILES>(p, b, hk, bh, split, row0, qc, o, m[qc], col_sum(l[qc]), lane);
  }
}

// Few rows (single tokens, beams): every wave owns all 16*QC rows and keys of its
// own, KT at a time, so k goes straight from memory into operands and v through
// a slice of LDS that only its wave touches: no barrier until the waves' results
// are joined, in one step.  Bound by the reading of k and v; a tile's loads are in
// flight while its predecessor is computed.  16 x 8 rows, 32768 keys, 32/8 heads of
// 128, bf16: 380 us = 5.6 TB/s (a copy reaches 5.0); 32 x 5 rows, 1000 keys, 8 heads
// of 64: 12.5 us, 4.0 TB/s, fp32 20.8 us, 4.8 TB/s; one row over 100 keys: 4.8 us, a
// launch.  Heads of 32 in bf16 reach half of that (6 rows of 64/8 heads, 31554 keys:
// 75 us, 2.6 TB/s): a head's row is half a cache line.
template <typename T, int DP, int QC, int NW, int KT>
__global__ void __launch_bounds__(NW * 64) attn_step_kernel(AttnParams p) {
  constexpr int SZ = AT<T>::SZ, PB = Pitch<T, DP>::B;
  constexpr int NCH = DP * SZ / 64, VR = DP * SZ / 16;
  constexpr int NV = KT * VR / 64;
  static_assert(KT * VR % 64 == 0, "tile divides over the wave");
  constexpr int NTILES = DP / 16;
  constexpr int kTiles = NW * KT * PB, kJoin = NW * QC * 16 * (DP + 4) * 4;
  __shared__ __align__(16) char smem[kTiles > kJoin ? kTiles : kJoin];
  __shared__ float sm[NW][QC * 16], sl[NW][QC * 16];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, l15 = lane & 15;
  const unsigned block = grid_block();
  if (block >= (unsigned)p.blocks) return;
  const int item = xcd_item(block, p.blocks);
  const int tile = item % p.tiles, rest = item / p.tiles;
  const int split = rest % p.nsplit, pair = rest / p.nsplit;
  const int b = pair % p.B, hk = pair / p.B, bh = b * p.Hkv + hk;
  const int db = p.D * SZ;
  const int s0 = split * p.kv_per_split;
  const int s1 = s0 + min(keys_of(p, b) - s0, p.kv_per_split);
  const char* kb = p.k + b * p.sk.b + hk * p.sk.h;
  const char* vb = p.v + b * p.sv.b + hk * p.sv.h;
  const uint8_t* mb = p.key_mask ? p.key_mask + (long long)b * p.S : nullptr;
  char* sv = smem + wave * KT * PB;

  const int row0 = tile * 16 * QC;
  uint4 qf[QC][NCH];
#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    const int r = row0 + qc * 16 + l15;
    const bool ok = r < p.rows;
    const int t = ok ? r / p.G : 0, gh = ok ? r % p.G : 0;
    const char* qr = p.q + b * p.sq.b + t * p.sq.t + (hk * p.G + gh) * p.sq.h;
#pragma unroll
    for (int c = 0; c < NCH; ++c) qf[qc][c] = load16(qr, c * 64 + g * 16, db, ok);
  }
  f32x4 o[NTILES][QC];
  float m[QC], l[QC];
#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    m[qc] = -INFINITY;
    l[qc] = 0.f;
#pragma unroll
    for (int n = 0; n < NTILES; ++n) o[n][qc] = (f32x4){0.f, 0.f, 0.f, 0.f};
  }

  uint4 kf[KT / 16][NCH], rv[NV];
  uint8_t mask = 0;  // lane i < KT: the mask byte of the tile's key i, a bit of every lane's `bits` below
  auto load_k = [&](int s) {
#pragma unroll
    for (int kt = 0; kt < KT / 16; ++kt) {
      const int r = s + kt * 16 + l15;
#pragma unroll
      for (int c = 0; c < NCH; ++c) kf[kt][c] = load16(kb + r * p.sk.t, c * 64 + g * 16, db, r < s1);
    }
    if (mb && lane < KT) mask = s + lane < s1 ? mb[s + lane] : 0;
  };
  auto load_v = [&](int s) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + j * 64, r = s + i / VR;
      rv[j] = load16(vb + r * p.sv.t, (i % VR) * 16, db, r < s1);
    }
  };
  const int first = s0 + wave * KT;
  if (first < s1) {
    load_k(first);
    load_v(first);
  }
  for (int s = first; s < s1; s += NW * KT) {
    f32x4 x[KT / 16][QC];
    const uint32_t bits = mb ? (uint32_t)__ballot(mask != 0) : 0xffffffffu;
#pragma unroll
    for (int kt = 0; kt < KT / 16; ++kt) {
#pragma unroll
      for (int qc = 0; qc < QC; ++qc) x[kt][qc] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        if (mb && !(bits >> (kt * 16 + l15) & 1)) kf[kt][c] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int qc = 0; qc < QC; ++qc) mma_chunk<T>(x[kt][qc], kf[kt][c], qf[qc][c]);
      }
      // -inf for keys left out, whatever q holds: a row without keys gives 0
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = kt * 16 + 4 * g + i;
        const bool key = s + at < s1 && (bits >> at & 1);
#pragma unroll
        for (int qc = 0; qc < QC; ++qc) x[kt][qc][i] = key ? x[kt][qc][i] : -INFINITY;
      }
    }
    if (s + NW * KT < s1) load_k(s + NW * KT);
    softmax_tile<T, DP, QC, KT, NTILES>(x, o, m, l, p.scale_log2);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + j * 64;
      if (mb && !(bits >> (i / VR) & 1)) rv[j] = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(sv + (i / VR) * PB + (i % VR) * 16) = rv[j];
    }
    if (s + NW * KT < s1) load_v(s + NW * KT);
    // the wave's own LDS accesses take effect in order; only the compiler has to keep them so
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    mma_tr<T, DP, QC, KT, NTILES>(o, sv, x, lane);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
  }

  // join the waves: their sums side by side in LDS, then 4 columns of a row a
  // thread, in wave order
  float* so = reinterpret_cast<float*>(smem);
  if (NW > 1) __syncthreads();
#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    l[qc] = col_sum(l[qc]);
    if (lane < 16) {
      sm[wave][qc * 16 + lane] = m[qc];
      sl[wave][qc * 16 + lane] = l[qc];
    }
    store_cols_f32<T, DP, NTILES, QC>(so + ((wave * QC + qc) * 16 + l15) * (DP + 4), o, qc, DP, lane);
  }
  __syncthreads();
  constexpr int per = DP / 4;
  for (int i = tid; i < QC * 16 * per; i += NW * 64) {
    const int r = i / per, d = i % per * 4, row = row0 + r;
    if (row >= p.rows || d >= p.D) continue;
    float mt = sm[0][r];
#pragma unroll
    for (int w = 1; w < NW; ++w) mt = fmaxf(mt, sm[w][r]);
    const float mu = mt == -INFINITY ? 0.f : mt;
    float lt = 0.f;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float by = exp2_fast(sm[w][r] - mu);
      lt += by * sl[w][r];
      x += *reinterpret_cast<const f32x4*>(so + (w * QC * 16 + r) * (DP + 4) + d) * by;
    }
    if (p.nsplit > 1) {
      const long long at = ((long long)bh * p.rows + row) * p.nsplit + split;
      *reinterpret_cast<f32x4*>(p.part_o + at * p.D + d) = x;
      if (d == 0) p.part_ml[at * 2] = mt, p.part_ml[at * 2 + 1] = lt;
    } else {
      const int t = row / p.G, hq = hk * p.G + row % p.G;
      x *= lt == 0.f ? 0.f : 1.f / lt;
      char* to = p.o + b * p.so.b + t * p.so.t + hq * p.so.h + d * SZ;
      if constexpr (AT<T>::BF) {
        const uint2 u = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
        *reinterpret_cast<uint2*>(to) = u;
        if (p.o_rest)
          *reinterpret_cast<uint2*>(p.o_rest + (((long long)bh * p.rows + row) * p.D + d) * 2) =
              make_uint2(rest_bf16(x[0], x[1], u.x), rest_bf16(x[2], x[3], u.y));
      } else {
        *reinterpret_cast<f32x4*>(to) = x;
      }
      if (d == 0 && p.lse) p.lse[((long long)b * p.Hq + hq) * p.Tq + t] = mu * kLn2 + logf(lt);
    }
  }
}

template <int QC, int NW, int KT>
hipError_t launch(const AttnParams& p, hipStream_t s) {
  hipLaunchKernelGGL((attn_fwd_kernel<ET, DP, QC, NW, KT>), grid_of(p.blocks), dim3(NW * 64), 0, s, p);
  return hipGetLastError();
}

template <int QC, int NW, int KT>
hipError_t launch_step(const AttnParams& p, hipStream_t s) {
  hipLaunchKernelGGL((attn_step_kernel<ET, DP, QC, NW, KT>), grid_of(p.blocks), dim3(NW * 64), 0, s, p);
  return hipGetLastError();
}

}  // namespace

#define DEC_FN2(bf, dp) attn_fwd_launch_##bf##_##dp
#define DEC_FN(bf, dp) DEC_FN2(bf, dp)
hipError_t DEC_FN(DEC_BF16, DEC_DP)(const AttnParams& p, hipStream_t s) {
  constexpr bool BF = DEC_BF16;
  constexpr int KT = fwd_key_tile(BF, DP), QC = fwd_columns(BF);
  switch (fwd_waves(BF, DP, p.rows)) {
    case 0:
      if constexpr (step_max_columns(BF, DP) == 2)
        if (step_columns(BF, DP, p.rows) == 2) return launch_step<2, 4, step_key_tile(BF)>(p, s);
      if constexpr (step_max_waves(BF, DP) == 8)
        if (step_waves(BF, DP, p.rows, p.S) == 8) return launch_step<1, 8, step_key_tile(BF)>(p, s);
      return launch_step<1, 4, step_key_tile(BF)>(p, s);
    case 4: return launch<QC, 4, KT>(p, s);
    default:
      if constexpr (fwd_max_waves(BF, DP) == 8) return launch<QC, 8, KT>(p, s);
      return hipErrorInvalidValue;
  }
}

}  // namespace lstm
