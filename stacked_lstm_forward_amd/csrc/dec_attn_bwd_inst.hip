// Attention over encoder outputs, gradients.  One translation unit per element
// type, padded head size (DEC_BF16, DEC_DP) and, where a wave's columns may be one
// or two groups, choice of these (DEC_NARROW).
//
// One launch of two kinds of workgroups, each recomputing the probabilities from
// q, k and lse: one kind owns keys and sums dk and dv over the rows, the other
// owns rows and sums dq over the keys.  The second pass over the scores costs two
// products of five more, and every sum stays in one wave's registers in a fixed
// order: no atomics, no partial dq in memory.  In one launch the tail of one kind
// is filled by the other.
//
// Bound by the latency of the dependent products of a tile at two or three waves a
// SIMD (matrix pipe busy 44 % of a working compute unit's time, vector pipe 45 %, LDS
// 43 %), and by the last round of workgroups: 4 x 2048 rows, 3001 keys at most, 12
// heads of 128, bf16 536 us, 740 TFLOP/s with the repeated products (the second ones
// of p and dz not counted).  32 x 200 rows, 777 keys, 4 key heads of 80: 80 us, the
// fixed cost of a workgroup being about as large as its 7 or 25 tiles.  fp32, 64 x 100
// rows, 120 keys at most, 8 heads of 64: 74 us, 55 % of it matrix products.  Where there
// are fewer workgroups than compute units, each still walks its whole other axis: 2 x
// 2000 rows, 200 keys, 2 heads of 64 take 72 us for 1.4 GFLOP.
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

#if DEC_NARROW
constexpr int C = 1, NW = 4, RT = 32, KT = 32, kPerSimd = kBwdNarrowWavesPerSimd;
constexpr bool kShort = false;
#else
constexpr int C = bwd_columns(DEC_BF16, DEC_DP), NW = bwd_waves(DEC_BF16, DEC_DP);
constexpr int RT = bwd_row_tile(DEC_BF16, DEC_DP), KT = bwd_key_tile(DEC_BF16, DEC_DP);
constexpr int kPerSimd = bwd_waves_per_simd(DEC_BF16, DEC_DP);
constexpr bool kShort = bwd_short(DEC_BF16, DEC_DP);
#endif
constexpr int NT = NW * 64;
constexpr int SZ = AT<ET>::SZ, PB = Pitch<ET, DP>::B;
constexpr int NCH = DP * SZ / 64, VR = DP * SZ / 16, NTILES = DP / 16;
// LDS: two buffers each, a tile is written while its predecessor is read.
struct KeySide {
  char q[2][RT * PB], d[2][RT * PB];
  float nl[2][RT], nd[2][RT];
  uint4 v[kShort ? NW * NCH * C * 64 : 1];  // the waves' own operands
};
struct RowSide {
  char k[2][KT * PB], v[2][KT * PB];
  float bias[2][KT];
};
constexpr int kShared = sizeof(KeySide) > sizeof(RowSide) ? sizeof(KeySide) : sizeof(RowSide);

// {-lse in base-2 units, -delta} of a row: {-inf, 0} where it has no key or lies
// past the list, so that p = exp2(z - inf) = 0.
__device__ __forceinline__ f32x2 row_stats(const AttnParams& p, int bh, int r) {
  return r < p.rows ? reinterpret_cast<const f32x2*>(p.stats)[(long long)bh * p.rows + r] : (f32x2){-INFINITY, 0.f};
}

// A workgroup's copy of RT rows of q and dout to LDS: load() issues the global
// reads a tile ahead, store() writes what arrived.  Each piece's addresses move by
// RT rows of the list (step, head of the group) a tile, without a division.
struct RowCopy {
  static constexpr int NV = (RT * VR + NT - 1) / NT;
  static constexpr bool EVEN = RT * VR % NT == 0;
  const char *aq[NV], *ad[NV];
  int g[NV];
  uint4 q[NV], d[NV];

  __device__ __forceinline__ int row(int tid, int j) const {
    const int i = tid + j * NT;
    return EVEN || i < RT * VR ? i / VR : 0;
  }
  __device__ __forceinline__ void init(const AttnParams& p, int b, int hk, int tid, int db) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = ((tid + j * NT) % VR) * 16, r = row(tid, j), t = r / p.G, col = c < db ? c : 0;
      g[j] = r % p.G;
      aq[j] = p.q + b * p.sq.b + t * p.sq.t + (hk * p.G + g[j]) * p.sq.h + col;
      ad[j] = p.dout + b * p.sdo.b + t * p.sdo.t + (hk * p.G + g[j]) * p.sdo.h + col;
    }
  }
  // the tile at row r0, the one after the last loaded
  __device__ __forceinline__ void load(const AttnParams& p, int r0, int tid) {
    if (r0 + RT <= p.rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        q[j] = *reinterpret_cast<const uint4*>(aq[j]);
        d[j] = *reinterpret_cast<const uint4*>(ad[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        q[j] = d[j] = make_uint4(0, 0, 0, 0);
        if (r0 + row(tid, j) < p.rows) {
          q[j] = *reinterpret_cast<const uint4*>(aq[j]);
          d[j] = *reinterpret_cast<const uint4*>(ad[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      g[j] += p.row_dg;
      const bool next = g[j] >= p.G;
      g[j] -= next ? p.G : 0;
      aq[j] += next ? p.row_q1 : p.row_q0;
      ad[j] += next ? p.row_d1 : p.row_d0;
    }
  }
  __device__ __forceinline__ void store(char* tq, char* td, int tid, int db) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * NT, c = (i % VR) * 16, a = (i / VR) * PB + c;
      if (db < DP * SZ && c >= db) q[j] = d[j] = make_uint4(0, 0, 0, 0);
      if (EVEN || i < RT * VR) {
        *reinterpret_cast<uint4*>(tq + a) = q[j];
        *reinterpret_cast<uint4*>(td + a) = d[j];
      }
    }
  }
};

// dk, dv: each wave owns 16*C keys (columns of S), the NW waves share the RT rows
// of a tile (q and dout) in LDS.  Waves without keys only copy.
__device__ __forceinline__ void key_side(const AttnParams& p, int item, char* smem) {
  KeySide& sh = *reinterpret_cast<KeySide*>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tile = item % p.kv_tiles, pair = item / p.kv_tiles;
  const int b = pair % p.B, hk = pair / p.B, bh = b * p.Hkv + hk;
  const int db = p.D * SZ;
  const int keys = keys_of(p, b);
  const int key0 = (tile * NW + wave) * 16 * C;
  const uint8_t* mb = p.key_mask ? p.key_mask + (long long)b * p.S : nullptr;

  // A key that the mask leaves out is read like any other: what it holds stays in
  // its own column, which is not stored.
  uint4 kf[C][NCH], vf[C][NCH];
  auto left = [&](int s) { return s < keys && (!mb || mb[s]); };
#pragma unroll
  for (int kc = 0; kc < C; ++kc) {
    const int s = key0 + kc * 16 + (lane & 15);
    const bool ok = s < keys;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      kf[kc][c] = load16(p.k + b * p.sk.b + s * p.sk.t + hk * p.sk.h, c * 64 + (lane >> 4) * 16, db, ok);
      const uint4 x = load16(p.v + b * p.sv.b + s * p.sv.t + hk * p.sv.h, c * 64 + (lane >> 4) * 16, db, ok);
      if constexpr (kShort)
        sh.v[((wave * NCH + c) * C + kc) * 64 + lane] = x;
      else
        vf[kc][c] = x;
    }
  }
  f32x4 dk[NTILES][C], dv[NTILES][C];
#pragma unroll
  for (int n = 0; n < NTILES; ++n)
#pragma unroll
    for (int kc = 0; kc < C; ++kc) dk[n][kc] = dv[n][kc] = (f32x4){0.f, 0.f, 0.f, 0.f};

  // keys past the last one leave their gradients zero
  const int rows = tile * NW * 16 * C < keys ? p.rows : 0;
  const bool live = key0 < keys;
  RowCopy cp;
  f32x2 st = {-INFINITY, 0.f};
  auto load = [&](int r0) {
    cp.load(p, r0, tid);
    if (tid < RT) st = row_stats(p, bh, r0 + tid);
  };
  auto store = [&](int buf) {
    cp.store(sh.q[buf], sh.d[buf], tid, db);
    if (tid < RT) {
      sh.nl[buf][tid] = st[0];
      sh.nd[buf][tid] = st[1];
    }
  };
  if (rows > 0) {
    cp.init(p, b, hk, tid, db);
    load(0);
    store(0);
  }
  __syncthreads();
  int buf = 0;
  for (int r0 = 0; r0 < rows; r0 += RT, buf ^= 1) {
    const bool more = r0 + RT < rows;
    if (more) load(r0 + RT);
    if (live) {
      f32x4 x[RT / 16][C], y[RT / 16][C];
      mma_rows0<ET, DP, C, RT>(x, sh.q[buf], kf, lane);
      if constexpr (!kShort) mma_rows0<ET, DP, C, RT>(y, sh.d[buf], vf, lane);
#pragma unroll
      for (int rt = 0; rt < RT / 16; ++rt) {
        const f32x4 nl = *reinterpret_cast<const f32x4*>(sh.nl[buf] + rt * 16 + (lane >> 4) * 4);
#pragma unroll
        for (int kc = 0; kc < C; ++kc)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[rt][kc][i] = exp2_fast(fmaf(x[rt][kc][i], p.scale_log2, nl[i]));
      }
      mma_tr<ET, DP, C, RT, NTILES>(dv, sh.d[buf], x, lane);
      if constexpr (kShort)
        mma_rows0_lds<ET, DP, C, RT>(y, sh.d[buf], reinterpret_cast<const uint4 (*)[C][64]>(sh.v + wave * NCH * C * 64), lane);
#pragma unroll
      for (int rt = 0; rt < RT / 16; ++rt) {
        const f32x4 nd = *reinterpret_cast<const f32x4*>(sh.nd[buf] + rt * 16 + (lane >> 4) * 4);
#pragma unroll
        for (int kc = 0; kc < C; ++kc) y[rt][kc] = (y[rt][kc] + nd) * x[rt][kc];
      }
      mma_tr<ET, DP, C, RT, NTILES>(dk, sh.q[buf], y, lane);
    }
    if (more) store(buf ^ 1);
    __syncthreads();
  }
#pragma unroll
  for (int kc = 0; kc < C; ++kc) {
    const int s = key0 + kc * 16 + (lane & 15);
    if (s >= p.S) continue;
    if (!left(s)) {
#pragma unroll
      for (int n = 0; n < NTILES; ++n) dk[n][kc] = dv[n][kc] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    store_cols<ET, DP, NTILES, C>(p.dk + b * p.sdk.b + s * p.sdk.t + hk * p.sdk.h, dk, kc, p.scale, p.D, lane);
    store_cols<ET, DP, NTILES, C>(p.dv + b * p.sdv.b + s * p.sdv.t + hk * p.sdv.h, dv, kc, 1.f, p.D, lane);
  }
}

// dq: each wave owns 16*C rows (columns of S^T), the waves share the KT keys of a
// tile (k and v) in LDS.  Waves without rows only copy.
__device__ __forceinline__ void row_side(const AttnParams& p, int item, char* smem) {
  RowSide& sh = *reinterpret_cast<RowSide*>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tile = item % p.tiles, pair = item / p.tiles;
  const int b = pair % p.B, hk = pair / p.B, bh = b * p.Hkv + hk;
  const int db = p.D * SZ;
  const int keys = keys_of(p, b);
  const uint8_t* mb = p.key_mask ? p.key_mask + (long long)b * p.S : nullptr;

  const int row0 = (tile * NW + wave) * 16 * C;
  uint4 qf[C][NCH], df[C][NCH];
  float nl[C], nd[C];
#pragma unroll
  for (int qc = 0; qc < C; ++qc) {
    const int r = row0 + qc * 16 + (lane & 15);
    const bool ok = r < p.rows;
    const int t = ok ? r / p.G : 0, hq = hk * p.G + (ok ? r % p.G : 0);
    const f32x2 st = row_stats(p, bh, r);
    nl[qc] = st[0];
    nd[qc] = st[1];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      qf[qc][c] = load16(p.q + b * p.sq.b + t * p.sq.t + hq * p.sq.h, c * 64 + (lane >> 4) * 16, db, ok);
      df[qc][c] = load16(p.dout + b * p.sdo.b + t * p.sdo.t + hq * p.sdo.h, c * 64 + (lane >> 4) * 16, db, ok);
    }
  }
  f32x4 dq[NTILES][C];
#pragma unroll
  for (int n = 0; n < NTILES; ++n)
#pragma unroll
    for (int qc = 0; qc < C; ++qc) dq[n][qc] = (f32x4){0.f, 0.f, 0.f, 0.f};

  const bool live = row0 < p.rows;
  TileCopy<ET, DP, KT, NT> ck, cv;
  uint8_t rb = 0;
  auto load = [&](int s) {
    ck.load(s, keys, mb, tid, db);
    cv.load(s, keys, nullptr, tid, db);
    if (tid < KT) rb = s + tid < keys ? (mb ? mb[s + tid] : 1) : 0;
  };
  auto store = [&](int buf, int s) {
    ck.store(sh.k[buf], s, keys, mb, tid, db, ck.m);
    cv.store(sh.v[buf], s, keys, mb, tid, db, ck.m);
    if (tid < KT) sh.bias[buf][tid] = rb ? 0.f : -INFINITY;
  };
  if (keys > 0) {
    ck.init(p.k + b * p.sk.b + hk * p.sk.h, p.sk.t, 0, tid, db);
    cv.init(p.v + b * p.sv.b + hk * p.sv.h, p.sv.t, 0, tid, db);
    load(0);
    store(0, 0);
  }
  __syncthreads();
  int buf = 0;
  for (int s = 0; s < keys; s += KT, buf ^= 1) {
    const bool more = s + KT < keys;
    if (more) load(s + KT);
    if (live) {
      f32x4 x[KT / 16][C], y[KT / 16][C];
#pragma unroll
      for (int kt = 0; kt < KT / 16; ++kt) {
        const f32x4 bias = *reinterpret_cast<const f32x4*>(sh.bias[buf] + kt * 16 + (lane >> 4) * 4);
#pragma unroll
        for (int qc = 0; qc < C; ++qc) {
          x[kt][qc] = bias;
          y[kt][qc] = (f32x4){nd[qc], nd[qc], nd[qc], nd[qc]};
        }
      }
      mma_rows<ET, DP, C, KT>(x, sh.k[buf], qf, lane);
      mma_rows<ET, DP, C, KT>(y, sh.v[buf], df, lane);
#pragma unroll
      for (int kt = 0; kt < KT / 16; ++kt)
#pragma unroll
        for (int qc = 0; qc < C; ++qc)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[kt][qc][i] = exp2_fast(fmaf(x[kt][qc][i], p.scale_log2, nl[qc])) * y[kt][qc][i];
      mma_tr<ET, DP, C, KT, NTILES>(dq, sh.k[buf], x, lane);
    }
    if (more) store(buf ^ 1, s + KT);
    __syncthreads();
  }
#pragma unroll
  for (int qc = 0; qc < C; ++qc) {
    const int r = row0 + qc * 16 + (lane & 15);
    if (r >= p.rows) continue;
    const int t = r / p.G, hq = hk * p.G + r % p.G;
    if (nl[qc] == -INFINITY) {  // no keys: 0, whatever q and dout hold
#pragma unroll
      for (int n = 0; n < NTILES; ++n) dq[n][qc] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    store_cols<ET, DP, NTILES, C>(p.dq + b * p.sdq.b + t * p.sdq.t + hq * p.sdq.h, dq, qc, p.scale, p.D, lane);
  }
}

__global__ void __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(kPerSimd)))
attn_bwd_kernel(AttnParams p) {
  __shared__ __align__(16) char smem[kShared];
  const unsigned block = grid_block();
  if (block >= (unsigned)p.blocks) return;
  const bool first = block < (unsigned)p.blocks_a;
  const int item = first ? xcd_item(block, p.blocks_a) : xcd_item(block - p.blocks_a, p.blocks - p.blocks_a);
  if (first != (p.rows_first != 0))
    key_side(p, item, smem);
  else
    row_side(p, item, smem);
}

}  // namespace

#if DEC_NARROW
#define DEC_FN2(bf, dp) attn_bwd_narrow_launch_##bf##_##dp
#else
#define DEC_FN2(bf, dp) attn_bwd_launch_##bf##_##dp
#endif
#define DEC_FN(bf, dp) DEC_FN2(bf, dp)
hipError_t DEC_FN(DEC_BF16, DEC_DP)(const AttnParams& p0, hipStream_t s) {
  AttnParams p = p0;
  const int dt = RT / p.G;
  p.row_dg = RT % p.G;
  p.row_q0 = dt * p.sq.t + p.row_dg * p.sq.h, p.row_q1 = p.row_q0 + p.sq.t - p.G * p.sq.h;
  p.row_d0 = dt * p.sdo.t + p.row_dg * p.sdo.h, p.row_d1 = p.row_d0 + p.sdo.t - p.G * p.sdo.h;
  p.tiles = (p.rows + NW * 16 * C - 1) / (NW * 16 * C);
  p.kv_tiles = (p.S + NW * 16 * C - 1) / (NW * 16 * C);
  // The row side, three products over the keys, goes first where its workgroups
  // take twice as long as the key side's, four over the rows (32 x 200 rows, 777
  // keys, D 80: 68 us, last 78); else last, where sentences that end early leave
  // short workgroups (4 x 2048 rows, 3001 keys, D 128: 463 us, first 505).
  p.rows_first = 3ll * p.S > 8ll * p.rows;
  p.blocks_a = p.B * p.Hkv * (p.rows_first ? p.tiles : p.kv_tiles);
  p.blocks = p.B * p.Hkv * (p.tiles + p.kv_tiles);
  hipLaunchKernelGGL(attn_bwd_kernel, grid_of(p.blocks), dim3(NT), 0, s, p);
  return hipGetLastError();
}

}  // namespace lstm
