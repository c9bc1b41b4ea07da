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

// Each wave owns 16*QC rows (columns of S^T), the workgroup's NW waves share
// the KT keys of a tile in LDS.
template <typename T, int DP, int QC, int NW, int KT>
__global__ void __launch_bounds__(NW * 64) attn_fwd_kernel(AttnParams p) {
  constexpr int SZ = AT<T>::SZ, NT = NW * 64, PB = Pitch<T, DP>::B;
  constexpr int NCH = DP * SZ / 64, VR = DP * SZ / 16;  // 16-byte pieces of a row
  constexpr int NV = KT * VR / NT;                      // pieces per thread and tile
  static_assert(KT * VR % NT == 0, "tile divides over the threads");
  constexpr int NTILES = DP / 16;
  __shared__ __align__(16) char sk[KT * PB];
  __shared__ __align__(16) char sv[KT * PB];
  __shared__ __align__(16) float sbias[KT];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int item = xcd_item(blockIdx.x, gridDim.x);
  const int tile = item % p.tiles, rest = item / p.tiles;
  const int split = rest % p.nsplit, bh = rest / p.nsplit;
  const int b = bh / p.Hkv, hk = bh % p.Hkv;
  const int db = p.D * SZ;

  const int s0 = split * p.kv_per_split;
  const int s1 = min(keys_of(p, b), s0 + p.kv_per_split);
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

  uint4 rk[NV], rv[NV];
  float rb = 0.f;
  auto load = [&](int s) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * NT, r = s + i / VR, c = (i % VR) * 16;
      const bool ok = r < s1 && (!mb || mb[r]);
      rk[j] = load16(kb + r * p.sk.t, c, db, ok);
      rv[j] = load16(vb + r * p.sv.t, c, db, ok);
    }
    if (tid < KT) rb = s + tid < s1 && (!mb || mb[s + tid]) ? 0.f : -INFINITY;
  };
  if (s0 < s1) load(s0);
  for (int s = s0; s < s1; s += KT) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * NT, a = (i / VR) * PB + (i % VR) * 16;
      *reinterpret_cast<uint4*>(sk + a) = rk[j];
      *reinterpret_cast<uint4*>(sv + a) = rv[j];
    }
    if (tid < KT) sbias[tid] = rb;
    __syncthreads();
    if (s + KT < s1) load(s + KT);

    f32x4 x[KT / 16][QC];
#pragma unroll
    for (int kt = 0; kt < KT / 16; ++kt) {
      const f32x4 bias = *reinterpret_cast<const f32x4*>(sbias + kt * 16 + (lane >> 4) * 4);
#pragma unroll
      for (int qc = 0; qc < QC; ++qc) x[kt][qc] = bias;
    }
    mma_rows<T, DP, QC, KT>(x, sk, qf, lane);
#pragma unroll
    for (int qc = 0; qc < QC; ++qc) {
      float mx = -INFINITY;
#pragma unroll
      for (int kt = 0; kt < KT / 16; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, x[kt][qc][i]);
      const float mn = fmaxf(m[qc], col_max(mx) * p.scale_log2);
      const float mu = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2_fast(m[qc] - mu);
      m[qc] = mn;
      float sum = 0.f;
#pragma unroll
      for (int kt = 0; kt < KT / 16; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = exp2_fast(fmaf(x[kt][qc][i], p.scale_log2, -mu));
          x[kt][qc][i] = e;
          sum += e;
        }
      l[qc] = l[qc] * alpha + sum;
#pragma unroll
      for (int n = 0; n < NTILES; ++n) o[n][qc] *= alpha;
    }
    mma_tr<T, DP, QC, KT, NTILES>(o, sv, x, lane);
  }

#pragma unroll
  for (int qc = 0; qc < QC; ++qc) {
    const float lt = col_sum(l[qc]);
    const int r = row0 + qc * 16 + (lane & 15);
    if (r >= p.rows) continue;
    if (p.nsplit > 1) {
      const long long at = ((long long)bh * p.rows + r) * p.nsplit + split;
      store_cols_f32<T, DP, NTILES, QC>(p.part_o + at * p.D, o, qc, p.D, lane);
      if (lane < 16) {
        p.part_ml[at * 2] = m[qc];
        p.part_ml[at * 2 + 1] = lt;
      }
    } else {
      const int t = r / p.G, hq = hk * p.G + r % p.G;
      store_cols<T, DP, NTILES, QC>(p.o + b * p.so.b + t * p.so.t + hq * p.so.h, o, qc, lt == 0.f ? 0.f : 1.f / lt,
                                    p.D, lane);
      if (lane < 16 && p.lse)
        p.lse[((long long)b * p.Hq + hq) * p.Tq + t] = (m[qc] == -INFINITY ? 0.f : m[qc]) * kLn2 + logf(lt);
    }
  }
}

template <int QC, int NW, int KT>
hipError_t launch(const AttnParams& p, hipStream_t s) {
  const long long n = (long long)p.B * p.Hkv * p.tiles * p.nsplit;
  hipLaunchKernelGGL((attn_fwd_kernel<ET, DP, QC, NW, KT>), dim3((unsigned)n), dim3(NW * 64), 0, s, p);
  return hipGetLastError();
}

}  // namespace

#define DEC_FN2(bf, dp) attn_fwd_launch_##bf##_##dp
#define DEC_FN(bf, dp) DEC_FN2(bf, dp)
hipError_t DEC_FN(DEC_BF16, DEC_DP)(const AttnParams& p, hipStream_t s) {
  constexpr int QC = DEC_BF16 ? 2 : 1;
  return launch<QC, 4, DEC_BF16 ? 64 : 32>(p, s);
}

}  // namespace lstm
