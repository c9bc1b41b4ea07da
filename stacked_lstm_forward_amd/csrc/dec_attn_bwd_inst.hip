// Attention over encoder outputs, gradients.  One translation unit per element
// type and padded head size (DEC_BF16, DEC_DP).
//
// Two kernels, each recomputing the probabilities from q, k and lse: one owns
// keys and sums dk and dv over the rows, one owns rows and sums dq over the
// keys.  The second pass over the scores costs two products of five more, and
// every sum stays in one wave's registers in a fixed order: no atomics, no
// partial dq in memory.
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

// Statistics of the rows of a tile: -lse in base-2 units (-inf where the row has
// no key, or lies past the list: p = exp2(z - inf) = 0) and -delta.
__device__ __forceinline__ void row_stats(const AttnParams& p, int b, int hk, int r, float& nlse, float& ndelta) {
  nlse = -INFINITY;
  ndelta = 0.f;
  if (r < p.rows) {
    const int t = r / p.G, hq = hk * p.G + r % p.G;
    const long long at = ((long long)b * p.Hq + hq) * p.Tq + t;
    const float ls = p.lse_in[at];
    nlse = ls == -INFINITY ? -INFINITY : -ls * kLog2e;
    ndelta = -p.delta[at];
  }
}

// dk, dv: each wave owns 16*KC keys (columns of S), the NW waves share the RT
// rows of a tile (q and dout) in LDS.
template <typename T, int DP, int KC, int NW, int RT>
__global__ void __launch_bounds__(NW * 64) attn_dkv_kernel(AttnParams p) {
  constexpr int SZ = AT<T>::SZ, NT = NW * 64, PB = Pitch<T, DP>::B;
  constexpr int NCH = DP * SZ / 64, VR = DP * SZ / 16;
  constexpr int NV = (RT * VR + NT - 1) / NT;
  constexpr int NTILES = DP / 16;
  __shared__ __align__(16) char sq[RT * PB];
  __shared__ __align__(16) char sd[RT * PB];
  __shared__ __align__(16) float snl[RT];
  __shared__ __align__(16) float snd[RT];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int item = xcd_item(blockIdx.x, gridDim.x);
  const int tile = item % p.kv_tiles, bh = item / p.kv_tiles;
  const int b = bh / p.Hkv, hk = bh % p.Hkv;
  const int db = p.D * SZ;
  const int keys = keys_of(p, b);
  const int key0 = (tile * NW + wave) * 16 * KC;
  const uint8_t* mb = p.key_mask ? p.key_mask + (long long)b * p.S : nullptr;

  uint4 kf[KC][NCH], vf[KC][NCH];
  float bias[KC];
#pragma unroll
  for (int kc = 0; kc < KC; ++kc) {
    const int s = key0 + kc * 16 + (lane & 15);
    const bool ok = s < keys && (!mb || mb[s]);
    bias[kc] = ok ? 0.f : -INFINITY;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      kf[kc][c] = load16(p.k + b * p.sk.b + s * p.sk.t + hk * p.sk.h, c * 64 + (lane >> 4) * 16, db, ok);
      vf[kc][c] = load16(p.v + b * p.sv.b + s * p.sv.t + hk * p.sv.h, c * 64 + (lane >> 4) * 16, db, ok);
    }
  }
  f32x4 dk[NTILES][KC], dv[NTILES][KC];
#pragma unroll
  for (int n = 0; n < NTILES; ++n)
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) dk[n][kc] = dv[n][kc] = (f32x4){0.f, 0.f, 0.f, 0.f};

  uint4 rq[NV], rd[NV];
  float rnl = 0.f, rnd = 0.f;
  auto load = [&](int r0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * NT, r = r0 + i / VR, c = (i % VR) * 16;
      const bool ok = i < RT * VR && r < p.rows;
      const int t = ok ? r / p.G : 0, hq = hk * p.G + (ok ? r % p.G : 0);
      rq[j] = load16(p.q + b * p.sq.b + t * p.sq.t + hq * p.sq.h, c, db, ok);
      rd[j] = load16(p.dout + b * p.sdo.b + t * p.sdo.t + hq * p.sdo.h, c, db, ok);
    }
    if (tid < RT) row_stats(p, b, hk, r0 + tid, rnl, rnd);
  };
  // keys past the last one leave their gradients zero
  const int rows = tile * NW * 16 * KC < keys ? p.rows : 0;
  if (rows > 0) load(0);
  for (int r0 = 0; r0 < rows; r0 += RT) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * NT, a = (i / VR) * PB + (i % VR) * 16;
      if (RT * VR % NT == 0 || i < RT * VR) {
        *reinterpret_cast<uint4*>(sq + a) = rq[j];
        *reinterpret_cast<uint4*>(sd + a) = rd[j];
      }
    }
    if (tid < RT) {
      snl[tid] = rnl;
      snd[tid] = rnd;
    }
    __syncthreads();
    if (r0 + RT < rows) load(r0 + RT);

    f32x4 x[RT / 16][KC], y[RT / 16][KC];
#pragma unroll
    for (int rt = 0; rt < RT / 16; ++rt) {
      const f32x4 nd = *reinterpret_cast<const f32x4*>(snd + rt * 16 + (lane >> 4) * 4);
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) {
        x[rt][kc] = (f32x4){bias[kc], bias[kc], bias[kc], bias[kc]};
        y[rt][kc] = nd;
      }
    }
    mma_rows<T, DP, KC, RT>(x, sq, kf, lane);
#pragma unroll
    for (int rt = 0; rt < RT / 16; ++rt) {
      const f32x4 nl = *reinterpret_cast<const f32x4*>(snl + rt * 16 + (lane >> 4) * 4);
#pragma unroll
      for (int kc = 0; kc < KC; ++kc)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[rt][kc][i] = exp2_fast(fmaf(x[rt][kc][i], p.scale_log2, nl[i]));
    }
    mma_tr<T, DP, KC, RT, NTILES>(dv, sd, x, lane);
    mma_rows<T, DP, KC, RT>(y, sd, vf, lane);
#pragma unroll
    for (int rt = 0; rt < RT / 16; ++rt)
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) y[rt][kc] *= x[rt][kc];
    mma_tr<T, DP, KC, RT, NTILES>(dk, sq, y, lane);
  }
#pragma unroll
  for (int kc = 0; kc < KC; ++kc) {
    const int s = key0 + kc * 16 + (lane & 15);
    if (s >= p.S) continue;
    const bool ok = bias[kc] == 0.f;
    store_cols<T, DP, NTILES, KC>(p.dk + b * p.sdk.b + s * p.sdk.t + hk * p.sdk.h, dk, kc, ok ? p.scale : 0.f, p.D,
                                  lane);
    store_cols<T, DP, NTILES, KC>(p.dv + b * p.sdv.b + s * p.sdv.t + hk * p.sdv.h, dv, kc, ok ? 1.f : 0.f, p.D, lane);
  }
}

// dq: each wave owns 16*QC rows (columns of S^T), the waves share the KT keys of
// a tile (k and v) in LDS.
template <typename T, int DP, int QC, int NW, int KT>
__global__ void __launch_bounds__(NW * 64) attn_dq_kernel(AttnParams p) {
  constexpr int SZ = AT<T>::SZ, NT = NW * 64, PB = Pitch<T, DP>::B;
  constexpr int NCH = DP * SZ / 64, VR = DP * SZ / 16;
  constexpr int NV = (KT * VR + NT - 1) / NT;
  constexpr int NTILES = DP / 16;
  __shared__ __align__(16) char sk[KT * PB];
  __shared__ __align__(16) char sv[KT * PB];
  __shared__ __align__(16) float sbias[KT];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int item = xcd_item(blockIdx.x, gridDim.x);
  const int tile = item % p.tiles, bh = item / p.tiles;
  const int b = bh / p.Hkv, hk = bh % p.Hkv;
  const int db = p.D * SZ;
  const int keys = keys_of(p, b);
  const char* kb = p.k + b * p.sk.b + hk * p.sk.h;
  const char* vb = p.v + b * p.sv.b + hk * p.sv.h;
  const uint8_t* mb = p.key_mask ? p.key_mask + (long long)b * p.S : nullptr;

  const int row0 = (tile * NW + wave) * 16 * QC;
  uint4 qf[QC][NCH], df[QC][NCH];
  float nl[QC], nd[QC];
#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    const int r = row0 + qc * 16 + (lane & 15);
    const bool ok = r < p.rows;
    const int t = ok ? r / p.G : 0, hq = hk * p.G + (ok ? r % p.G : 0);
    row_stats(p, b, hk, r, nl[qc], nd[qc]);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      qf[qc][c] = load16(p.q + b * p.sq.b + t * p.sq.t + hq * p.sq.h, c * 64 + (lane >> 4) * 16, db, ok);
      df[qc][c] = load16(p.dout + b * p.sdo.b + t * p.sdo.t + hq * p.sdo.h, c * 64 + (lane >> 4) * 16, db, ok);
    }
  }
  f32x4 dq[NTILES][QC];
#pragma unroll
  for (int n = 0; n < NTILES; ++n)
#pragma unroll
    for (int qc = 0; qc < QC; ++qc) dq[n][qc] = (f32x4){0.f, 0.f, 0.f, 0.f};

  uint4 rk[NV], rv[NV];
  float rb = 0.f;
  auto load = [&](int s) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * NT, r = s + i / VR, c = (i % VR) * 16;
      const bool ok = i < KT * VR && r < keys && (!mb || mb[r]);
      rk[j] = load16(kb + r * p.sk.t, c, db, ok);
      rv[j] = load16(vb + r * p.sv.t, c, db, ok);
    }
    if (tid < KT) rb = s + tid < keys && (!mb || mb[s + tid]) ? 0.f : -INFINITY;
  };
  if (keys > 0) load(0);
  for (int s = 0; s < keys; s += KT) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * NT, a = (i / VR) * PB + (i % VR) * 16;
      if (KT * VR % NT == 0 || i < KT * VR) {
        *reinterpret_cast<uint4*>(sk + a) = rk[j];
        *reinterpret_cast<uint4*>(sv + a) = rv[j];
      }
    }
    if (tid < KT) sbias[tid] = rb;
    __syncthreads();
    if (s + KT < keys) load(s + KT);

    f32x4 x[KT / 16][QC], y[KT / 16][QC];
#pragma unroll
    for (int kt = 0; kt < KT / 16; ++kt) {
      const f32x4 bias = *reinterpret_cast<const f32x4*>(sbias + kt * 16 + (lane >> 4) * 4);
#pragma unroll
      for (int qc = 0; qc < QC; ++qc) {
        x[kt][qc] = bias;
        y[kt][qc] = (f32x4){nd[qc], nd[qc], nd[qc], nd[qc]};
      }
    }
    mma_rows<T, DP, QC, KT>(x, sk, qf, lane);
    mma_rows<T, DP, QC, KT>(y, sv, df, lane);
#pragma unroll
    for (int kt = 0; kt < KT / 16; ++kt)
#pragma unroll
      for (int qc = 0; qc < QC; ++qc)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[kt][qc][i] = exp2_fast(fmaf(x[kt][qc][i], p.scale_log2, nl[qc])) * y[kt][qc][i];
    mma_tr<T, DP, QC, KT, NTILES>(dq, sk, x, lane);
  }
#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    const int r = row0 + qc * 16 + (lane & 15);
    if (r >= p.rows) continue;
    const int t = r / p.G, hq = hk * p.G + r % p.G;
    store_cols<T, DP, NTILES, QC>(p.dq + b * p.sdq.b + t * p.sdq.t + hq * p.sdq.h, dq, qc, p.scale, p.D, lane);
  }
}

}  // namespace

#define DEC_FN2(bf, dp) attn_bwd_launch_##bf##_##dp
#define DEC_FN(bf, dp) DEC_FN2(bf, dp)
hipError_t DEC_FN(DEC_BF16, DEC_DP)(const AttnParams& p, hipStream_t s) {
  constexpr int C = bwd_columns(DEC_BF16, DEC_DP), T = 32;
  if (p.S > 0) {
    const long long n = (long long)p.B * p.Hkv * p.kv_tiles;
    hipLaunchKernelGGL((attn_dkv_kernel<ET, DP, C, 4, T>), dim3((unsigned)n), dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const long long n = (long long)p.B * p.Hkv * p.tiles;
  hipLaunchKernelGGL((attn_dq_kernel<ET, DP, C, 4, T>), dim3((unsigned)n), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace lstm
