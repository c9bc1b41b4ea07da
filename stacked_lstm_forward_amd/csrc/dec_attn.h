// Attention over encoder outputs: parameters and device helpers shared by its
// forward, single-step and backward kernels (gfx950 / CDNA4).
//
// Rows.  The G = Hq/Hkv query heads of one key head and the Tq steps form one
// list of rows, r = t*G + g, so that shared heads and beams read k and v once.
//
// Products.  Every kernel forms the scores transposed where its wave owns query
// rows (S^T = K Q^T, "columns are queries") and untransposed where it owns keys
// (S = Q K^T, "columns are keys"): either way the 16x16 output of one MFMA
// (lane l: column l%16, rows 4*(l/16)+i) is, after the softmax and the split below,
// already the B operand of the next product, whose sum runs over those rows.
// The order of a product's sum is free, so the k-slots of that operand are
// taken as they lie: for bf16 (16x16x32) lane group g holds rows 4g..4g+3 of two
// 16-row tiles, for fp32 (16x16x4, step i) row 4g+i.  The A operand of that
// product is read with the same rows: transposed 8-byte LDS reads
// (ds_read_b64_tr_b16) in bf16, plain row reads in fp32.  The scores never
// leave registers.
//
// Operands of the first products are 16 bytes per lane and 64-byte chunk of a
// row: chunk c, lane group g holds bytes 64c+16g .. +15 (8 bf16 or 4 fp32
// values) of row l%16, for A and B alike.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dec_grid.h"
#include "lstm_common.h"

namespace lstm {

struct AttnStride {
  long long b, t, h;  // bytes
};

struct AttnParams {
  const char *q, *k, *v, *o_in, *dout;
  char *o, *dq, *dk, *dv;
  char* o_rest;          // bf16: what o's rounding leaves, [B*Hkv][rows][D]; may be null
  float* lse;            // [B][Hq][Tq]; the forward's may be null
  const float* lse_in;   // the backward's
  const int32_t* kv_len;
  const uint8_t* key_mask;
  AttnStride sq, sk, sv, so, sdo, sdq, sdk, sdv;
  int B, Tq, S, Hq, Hkv, G, D;
  int rows;              // Tq * G
  int tiles;             // row tiles per (sentence, key head)
  int nsplit, kv_per_split;
  int blocks;            // workgroups of the launch
  int kv_tiles;          // backward: key tiles per (sentence, key head)
  float scale, scale_log2;  // scale, scale * log2(e)
  float* part_o;         // nsplit > 1: [B*Hkv*rows][nsplit][D] unnormalised
  float* part_ml;        // [B*Hkv*rows][nsplit][2]: maximum (base-2 units) and sum
  float* stats;          // backward: [B*Hkv][rows][2], -lse (base-2 units) and -delta
  int rows_first, blocks_a;  // backward: workgroups that own rows go first; workgroups that go first
  int row_dg;            // backward: a tile of rows ahead, heads of the group and bytes of q and dout
  long long row_q0, row_q1, row_d0, row_d1;  // (.1: where the head passes the group's end)
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

template <typename T>
struct AT;
template <>
struct AT<uint16_t> {  // bfloat16
  static constexpr int SZ = 2;
  static constexpr bool BF = true;
};
template <>
struct AT<float> {
  static constexpr int SZ = 4;
  static constexpr bool BF = false;
};

// acc += A(16 rows x one 64-byte chunk) * B(chunk x 16 columns)
template <typename T>
__device__ __forceinline__ void mma_chunk(f32x4& acc, const uint4& a, const uint4& b) {
  if constexpr (AT<T>::BF) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc,
                                                  0, 0, 0);
  } else {
    const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[j], fb[j], acc, 0, 0, 0);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 r = __builtin_convertvector((f32x2){lo, hi}, bf16x2);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __builtin_bit_cast(float, u & 0xffff0000u); }

// The value of lane l^32 beside this lane's own (in either order); lane l^16 likewise.
// (The halves go through plain variables: __builtin_bit_cast of a vector element reads element 0.)
struct Pair {
  float x, y;
};
__device__ __forceinline__ Pair swap32(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t x = r[0], y = r[1];
  return {__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)};
}
__device__ __forceinline__ Pair swap16(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t x = r[0], y = r[1];
  return {__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)};
}

// Maximum and sum over the four lane groups of one column (lanes l, l^16, l^32, l^48).
__device__ __forceinline__ float col_max(float v) {
  const Pair a = swap32(v);
  const Pair b = swap16(fmaxf(a.x, a.y));
  return fmaxf(b.x, b.y);
}
__device__ __forceinline__ float col_sum(float v) {
  const Pair a = swap32(v);
  const Pair b = swap16(a.x + a.y);
  return b.x + b.y;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Row pitch of an LDS tile of DP columns.  The 16-byte row reads want successive
// rows 4 banks apart, the transposed 8-byte reads (4 rows x 32 bytes per 16
// lanes) 8 banks apart; the pitch serves the second, since the first keep 8
// rows on distinct banks either way.
template <typename T, int DP>
struct Pitch {
  static constexpr int B = DP * AT<T>::SZ + (AT<T>::BF ? 32 : 16);
};

// The A operands of one product over 32 (bf16) or 16 (fp32) rows of an LDS tile,
// transposed: output row m of MFMA tile n is column out_col(n, m) of the tile.
// bf16: 16 columns a tile.  fp32: W = 4 (2 where the columns are no multiple of
// 64) tiles at a time from one W-float read, tile t of block u holding columns
// 16*W*u + W*m + t.
template <typename T, int DP>
struct TrA {
  static constexpr int W = AT<T>::BF ? 1 : (DP % 64 == 0 ? 4 : 2);
  static constexpr int NT = DP / 16;  // MFMA tiles
};

__device__ __forceinline__ s16x4 lds_tr4(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)(p));
}

// acc[n][qc] += tile(32 rows, transposed) * (hi + lo)[..][qc] for all column tiles n;
// hi and lo hold the packed values of two 16-row tiles.
template <typename T, int DP, int QC, int NTILES>
__device__ __forceinline__ void mma_tr_bf16(f32x4 (&acc)[NTILES][QC], const char* tile, const uint4 (&hi)[QC],
                                            const uint4 (&lo)[QC], int lane) {
  constexpr int PB = Pitch<T, DP>::B;
  const char* base = tile + (lane >> 2) * PB + (lane & 3) * 8;
#pragma unroll
  for (int n = 0; n < NTILES; ++n) {
    const s16x4 x = lds_tr4(base + n * 32);
    const s16x4 y = lds_tr4(base + n * 32 + 16 * PB);
    const bf16x8 a = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
    for (int qc = 0; qc < QC; ++qc) {
      acc[n][qc] =
          __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, hi[qc]), acc[n][qc], 0, 0, 0);
      acc[n][qc] =
          __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, lo[qc]), acc[n][qc], 0, 0, 0);
    }
  }
}

// acc += (KT rows of `tile`, transposed) * p in fp32.  A tile's sum is taken by itself
// and then added, so that a long sum takes KT roundings and one for each tile, not one
// for each row (dv of 20000 rows: 2-norm error 2.6e-6 row by row).
template <int DP, int QC, int KT, int NTILES>
__device__ __forceinline__ void mma_tr_f32(f32x4 (&acc)[NTILES][QC], const char* tile, const f32x4 (&p)[KT / 16][QC],
                                           int lane) {
  constexpr int PB = Pitch<float, DP>::B;
  constexpr int W = TrA<float, DP>::W;
  typedef float Wide __attribute__((ext_vector_type(W)));
  const char* base = tile + 4 * (lane >> 4) * PB + (lane & 15) * W * 4;
#pragma unroll
  for (int u = 0; u < NTILES / W; ++u) {
    f32x4 sum[W][QC];
#pragma unroll
    for (int t = 0; t < W; ++t)
#pragma unroll
      for (int qc = 0; qc < QC; ++qc) sum[t][qc] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kt = 0; kt < KT / 16; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Wide a = *reinterpret_cast<const Wide*>(base + (kt * 16 + i) * PB + u * 16 * W * 4);
#pragma unroll
        for (int t = 0; t < W; ++t)
#pragma unroll
          for (int qc = 0; qc < QC; ++qc)
            sum[t][qc] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[t], p[kt][qc][i], sum[t][qc], 0, 0, 0);
      }
#pragma unroll
    for (int t = 0; t < W; ++t)
#pragma unroll
      for (int qc = 0; qc < QC; ++qc) acc[u * W + t][qc] += sum[t][qc];
  }
}

// x and y less the rounded values that u holds
__device__ __forceinline__ uint32_t rest_bf16(float x, float y, uint32_t u) {
  return pack_bf16(x - bf16_lo(u), y - bf16_hi(u));
}

// acc += (rows of `tile`, KT of them, transposed) * p, p in score layout
// [KT/16][QC], fp32.  For bf16 products p is the sum of two bf16 values, its
// rounding and the rounding of what that leaves (together within 2^-16 of p), and
// each takes a product of its own.  One rounding of p (2^-8) would add an error as
// large as the outputs' own rounding: 2-norm errors of o, dq, dk, dv against 64 bits
// 0.0023, 0.0024-0.0025, 0.0024, 0.0023 instead of the 0.0017 that the outputs'
// rounding alone gives.  The second product costs nothing where reading k and v is the
// bound (16 x 8 rows, 32768 keys: 384 us either way), 15 % where latency is (64 x 200
// rows, 331 keys: 16.3 and 19.2 us) and 25 % of the longest cases (8 x 2048 rows, 4096
// keys, 32 heads of 128: 1.22 and 1.52 ms; the training step of 4 x 2048 rows, 3001
// keys, 12 heads of 128: 599 and 737 us).
template <typename T, int DP, int QC, int KT, int NTILES>
__device__ __forceinline__ void mma_tr(f32x4 (&acc)[NTILES][QC], const char* tile, const f32x4 (&p)[KT / 16][QC],
                                       int lane) {
  if constexpr (AT<T>::BF) {
    constexpr int PB = Pitch<T, DP>::B;
#pragma unroll
    for (int ks = 0; ks < KT / 32; ++ks) {
      uint4 hi[QC], lo[QC];
#pragma unroll
      for (int qc = 0; qc < QC; ++qc) {
        const f32x4 x = p[2 * ks][qc], y = p[2 * ks + 1][qc];
        const uint4 h = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(y[0], y[1]),
                                   pack_bf16(y[2], y[3]));
        hi[qc] = h;
        lo[qc] = make_uint4(rest_bf16(x[0], x[1], h.x), rest_bf16(x[2], x[3], h.y), rest_bf16(y[0], y[1], h.z),
                            rest_bf16(y[2], y[3], h.w));
      }
      mma_tr_bf16<T, DP, QC, NTILES>(acc, tile + ks * 32 * PB, hi, lo, lane);
    }
  } else {
    mma_tr_f32<DP, QC, KT, NTILES>(acc, tile, p, lane);
  }
}

// s[kt][qc] += rows of `tile` (KT of them) * frag columns
template <typename T, int DP, int QC, int KT>
__device__ __forceinline__ void mma_rows(f32x4 (&s)[KT / 16][QC], const char* tile,
                                         const uint4 (&b)[QC][DP * AT<T>::SZ / 64], int lane) {
  constexpr int PB = Pitch<T, DP>::B;
  constexpr int NCH = DP * AT<T>::SZ / 64;
  const char* base = tile + (lane & 15) * PB + (lane >> 4) * 16;
#pragma unroll
  for (int kt = 0; kt < KT / 16; ++kt)
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const uint4 a = *reinterpret_cast<const uint4*>(base + kt * 16 * PB + c * 64);
#pragma unroll
      for (int qc = 0; qc < QC; ++qc) mma_chunk<T>(s[kt][qc], a, b[qc][c]);
    }
}

// Writes one column's results (d values of lane group g) of an accumulator laid
// out by mma_tr to a row of D values, scaled, as T; what a rounding leaves to `rest`
// where that is given.
template <typename T, int DP, int NTILES, int QC>
__device__ __forceinline__ void store_cols(char* row, const f32x4 (&acc)[NTILES][QC], int qc, float by, int D,
                                           int lane, char* rest = nullptr) {
  constexpr int W = TrA<T, DP>::W;
  const int g = lane >> 4;
  if constexpr (AT<T>::BF) {
#pragma unroll
    for (int n = 0; n < NTILES; ++n) {
      const int d = n * 16 + 4 * g;
      if (d < D) {
        const f32x4 x = acc[n][qc] * by;
        const uint2 u = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
        *reinterpret_cast<uint2*>(row + d * 2) = u;
        if (rest)
          *reinterpret_cast<uint2*>(rest + d * 2) = make_uint2(rest_bf16(x[0], x[1], u.x), rest_bf16(x[2], x[3], u.y));
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < NTILES / W; ++u) {
      // lane group g: rows m = 4g+i of tiles t: columns 16Wu + 4Wg + (W i + t), 4W in a row
      float x[4 * W];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < W; ++t) x[W * i + t] = acc[u * W + t][qc][i] * by;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int d = 16 * W * u + 4 * W * g + 4 * j;
        if (d < D)
          *reinterpret_cast<f32x4*>(row + d * 4) = (f32x4){x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
      }
    }
  }
}

// fp32 copy of the same (partial results of a split)
template <typename T, int DP, int NTILES, int QC>
__device__ __forceinline__ void store_cols_f32(float* row, const f32x4 (&acc)[NTILES][QC], int qc, int D, int lane) {
  constexpr int W = TrA<T, DP>::W;
  const int g = lane >> 4;
#pragma unroll
  for (int u = 0; u < NTILES / W; ++u) {
    float x[4 * W];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < W; ++t) x[W * i + t] = acc[u * W + t][qc][i];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const int d = 16 * W * u + 4 * W * g + 4 * j;
      if (d < D) *reinterpret_cast<f32x4*>(row + d) = (f32x4){x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
    }
  }
}

// A 16-byte piece of row r of a row list, zero outside (columns >= D, !ok).
__device__ __forceinline__ uint4 load16(const char* row, int byte, int dbytes, bool ok) {
  return ok && byte < dbytes ? *reinterpret_cast<const uint4*>(row + byte) : make_uint4(0, 0, 0, 0);
}

// Zero-initialised first products: s[kt][qc] = rows of `tile` * frag columns.
template <typename T, int DP, int QC, int KT>
__device__ __forceinline__ void mma_rows0(f32x4 (&s)[KT / 16][QC], const char* tile,
                                          const uint4 (&b)[QC][DP * AT<T>::SZ / 64], int lane) {
#pragma unroll
  for (int kt = 0; kt < KT / 16; ++kt)
#pragma unroll
    for (int qc = 0; qc < QC; ++qc) s[kt][qc] = (f32x4){0.f, 0.f, 0.f, 0.f};
  mma_rows<T, DP, QC, KT>(s, tile, b, lane);
}

// The same with the columns' operands in LDS.
template <typename T, int DP, int QC, int KT>
__device__ __forceinline__ void mma_rows0_lds(f32x4 (&s)[KT / 16][QC], const char* tile,
                                              const uint4 (*b)[QC][64], int lane) {
  constexpr int PB = Pitch<T, DP>::B;
  const char* base = tile + (lane & 15) * PB + (lane >> 4) * 16;
#pragma unroll
  for (int kt = 0; kt < KT / 16; ++kt)
#pragma unroll
    for (int qc = 0; qc < QC; ++qc) s[kt][qc] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < DP * AT<T>::SZ / 64; ++c) {
    uint4 f[QC];
#pragma unroll
    for (int qc = 0; qc < QC; ++qc) f[qc] = b[c][qc][lane];
#pragma unroll
    for (int kt = 0; kt < KT / 16; ++kt) {
      const uint4 a = *reinterpret_cast<const uint4*>(base + kt * 16 * PB + c * 64);
#pragma unroll
      for (int qc = 0; qc < QC; ++qc) mma_chunk<T>(s[kt][qc], a, f[qc]);
    }
  }
}

// A workgroup's copy of KT rows of one tensor to LDS, in two halves: load() issues
// the global reads a tile ahead, store() writes what arrived.  Rows at or past
// `end` (read as row end-1), columns at or past D and rows whose key mask byte
// (read beside them) is 0 are written as zeros.  Full tiles are addressed by a
// running pointer.
template <typename T, int DP, int KT, int NT>
struct TileCopy {
  static constexpr int SZ = AT<T>::SZ, PB = Pitch<T, DP>::B, VR = DP * SZ / 16;
  static constexpr int NV = (KT * VR + NT - 1) / NT;
  static constexpr bool EVEN = KT * VR % NT == 0;
  const char* at[NV];  // this thread's pieces of the tile at key `s`
  uint4 x[NV];
  uint8_t m[NV];
  const char* base;
  long long step;

  __device__ __forceinline__ void init(const char* b, long long st, int s, int tid, int db) {
    base = b;
    step = st;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * NT, c = (i % VR) * 16;
      at[j] = b + (s + (EVEN || i < KT * VR ? i / VR : 0)) * st + (c < db ? c : 0);
    }
  }
  // loads the tile at s, which is the one init() named or the one after the last loaded
  __device__ __forceinline__ void load(int s, int end, const uint8_t* mb, int tid, int db) {
    if (s + KT <= end) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        x[j] = *reinterpret_cast<const uint4*>(at[j]);
        at[j] += KT * step;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = tid + j * NT, c = (i % VR) * 16;
        const int r = min(s + (EVEN || i < KT * VR ? i / VR : 0), end - 1);
        x[j] = *reinterpret_cast<const uint4*>(base + r * step + (c < db ? c : 0));
      }
    }
    if (mb) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = tid + j * NT;
        m[j] = mb[min(s + (EVEN || i < KT * VR ? i / VR : 0), end - 1)];
      }
    }
  }
  // (`m` are the mask bytes of these rows, which another tensor's copy may have read)
  __device__ __forceinline__ void store(char* to, int s, int end, const uint8_t* mb, int tid, int db,
                                        const uint8_t (&m)[NV]) {
    if (s + KT > end) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (s + (tid + j * NT) / VR >= end) x[j] = make_uint4(0, 0, 0, 0);
    }
    if (mb) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (!m[j]) x[j] = make_uint4(0, 0, 0, 0);
    }
    if (db < DP * SZ) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (((tid + j * NT) % VR) * 16 >= db) x[j] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * NT, a = (i / VR) * PB + (i % VR) * 16;
      if (EVEN || i < KT * VR) *reinterpret_cast<uint4*>(to + a) = x[j];
    }
  }
};

// Number of keys of sentence b before the key mask.
__device__ __forceinline__ int keys_of(const AttnParams& p, int b) {
  int n = p.S;
  if (p.kv_len) n = min(max(p.kv_len[b], 0), p.S);
  return n;
}

// Block number -> work item such that the items of one XCD (blocks go round
// robin over the 8 XCDs) are neighbours and share their k and v in its L2.  The
// sentences follow each other within a head, so that every XCD gets short and
// long ones.
__device__ __forceinline__ int xcd_item(int block, int n) {
  const int per = n >> 3, extra = n & 7, x = block & 7, slot = block >> 3;
  return x * per + min(x, extra) + slot;
}

}  // namespace lstm
