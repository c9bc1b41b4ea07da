// One step of beam search (include/decoder/lstm_dec.h): two launches.
//
//   rows   one wave per part of a beam's row of logits: reads it once, keeps the
//          part's sum of exponentials and, per lane, the best value seen with the
//          first 16-byte vector that holds it; then takes the part's K best in
//          the order (value falling, index rising).  These lie in the K lanes
//          whose best come first in that order, and none is below the last of
//          the K lanes' bests: the wave rereads these lanes' vectors only and
//          keeps what reaches that value.
//   join   one sentence per workgroup (several where the states are large, each
//          joining again): a wave per beam takes its log-sum-exp in 64 bits and
//          its K best from its parts, one wave the K best of all by rank, and all
//          copy the chosen states.
//
// The order of every sum and every comparison is by index in the row, never by
// address: beams with equal rows get equal sums, and their ties stay ties.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <climits>
#include <cmath>

#include "decoder/lstm_dec.h"  // include/ is on the include path
#include "lstm_common.h"

namespace lstm {
namespace {

constexpr int kMaxK = 16;
constexpr int kMaxParts = 64;
constexpr int kVecsPerLane = 64;  // of one part: an extraction rereads one lane's with one load
constexpr int kMaxV = 1 << 20;    // kMaxParts * 64 * kVecsPerLane vectors of four values

struct BeamParams {
  const void* logits;
  const float* scores;
  const uint8_t* finished;
  const int32_t* lengths;
  int32_t *tokens, *parents;
  float* scores_out;
  uint8_t* finished_out;
  int32_t* lengths_out;
  const char *h, *c;
  char *h_out, *c_out;
  int B, K, V, eos, L, H, h_size;
  float alpha;
  long long stride;      // elements between rows
  int parts, vecs;       // parts of a row, 16-byte vectors of a part
  int copies;            // workgroups per sentence of the join
  int vec_copy;          // state rows are whole aligned 16-byte vectors
  double* part_sum;      // [B*K][parts]
  float* part_m;         // [B*K][parts]
  float* part_val;       // [B*K][parts][K]
  int* part_idx;
};

// ---- wave reductions: every lane gets the result -----------------------------
template <int CTRL>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false);
}
constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ float wave_max(float x) {
  auto f = [](int v) { return __builtin_bit_cast(float, v); };
  auto u = [](float v) { return __builtin_bit_cast(int, v); };
  x = fmaxf(x, f(dpp<kXor1>(u(x))));
  x = fmaxf(x, f(dpp<kXor2>(u(x))));
  x = fmaxf(x, f(dpp<kHalfMirror>(u(x))));
  x = fmaxf(x, f(dpp<kMirror>(u(x))));
  const auto a = __builtin_amdgcn_permlane16_swap(u(x), u(x), false, false);
  const int a0 = a[0], a1 = a[1];
  x = fmaxf(f(a0), f(a1));
  const auto b = __builtin_amdgcn_permlane32_swap(u(x), u(x), false, false);
  const int b0 = b[0], b1 = b[1];
  return fmaxf(f(b0), f(b1));
}
__device__ __forceinline__ int wave_min(int x) {
  x = min(x, dpp<kXor1>(x));
  x = min(x, dpp<kXor2>(x));
  x = min(x, dpp<kHalfMirror>(x));
  x = min(x, dpp<kMirror>(x));
  auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = min((int)a[0], (int)a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return min((int)b[0], (int)b[1]);
}
// The lane that holds the largest v, of equals the lowest idx.  v is no NaN.
__device__ __forceinline__ int wave_best(float v, int idx) {
  const float mx = wave_max(v);
  const bool top = v == mx;
  unsigned long long who = __ballot(top);
  if (__popcll(who) > 1) {
    const int mn = wave_min(top ? idx : INT_MAX);
    who = __ballot(top && idx == mn);
  }
  return __builtin_amdgcn_readfirstlane(__ffsll((long long)who) - 1);
}
__device__ __forceinline__ float lane_f(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// ---- rows ---------------------------------------------------------------------
// 16 bytes at an address that is a multiple of the element's size only
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

template <bool BF>
struct Row;
template <>
struct Row<true> {
  static constexpr int VE = 8;
  typedef uint16_t E;
  typedef u32x4_a2 Raw;
  static __device__ __forceinline__ float value(E e) { return __builtin_bit_cast(float, (uint32_t)e << 16); }
  static __device__ __forceinline__ void split(const Raw& u, float (&x)[VE]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = u[j];
      x[2 * j] = __builtin_bit_cast(float, w << 16);
      x[2 * j + 1] = __builtin_bit_cast(float, w & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Raw raw(const void* base, int i) {
    return *reinterpret_cast<const Raw*>(static_cast<const E*>(base) + i);
  }
  static __device__ __forceinline__ void load(const void* base, int i, int n, float pad, float (&x)[VE]);
};
template <>
struct Row<false> {
  static constexpr int VE = 4;
  typedef float E;
  typedef u32x4_a4 Raw;
  static __device__ __forceinline__ float value(E e) { return e; }
  static __device__ __forceinline__ void split(const Raw& u, float (&x)[VE]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = u[j];
      x[j] = __builtin_bit_cast(float, w);
    }
  }
  static __device__ __forceinline__ Raw raw(const void* base, int i) {
    return *reinterpret_cast<const Raw*>(static_cast<const E*>(base) + i);
  }
  static __device__ __forceinline__ void load(const void* base, int i, int n, float pad, float (&x)[VE]);
};
// values i .. i+VE-1 of a row of n; past its end `pad`
template <typename R>
__device__ __forceinline__ void load_row(const void* base, int i, int n, float pad, float (&x)[R::VE]) {
  if (i + R::VE <= n) {
    R::split(R::raw(base, i), x);
    return;
  }
#pragma unroll
  for (int j = 0; j < R::VE; ++j) {
    x[j] = pad;
    if (i + j < n) x[j] = R::value(static_cast<const typename R::E*>(base)[i + j]);
  }
}
__device__ __forceinline__ void Row<true>::load(const void* base, int i, int n, float pad, float (&x)[VE]) {
  load_row<Row<true>>(base, i, n, pad, x);
}
__device__ __forceinline__ void Row<false>::load(const void* base, int i, int n, float pad, float (&x)[VE]) {
  load_row<Row<false>>(base, i, n, pad, x);
}

// log2(e) as a sum of two floats
constexpr float kL2eHi = 1.44268798828125f;
constexpr float kL2eLo = 7.052607713387005e-06f;
constexpr float kLowest = -3.402823466e38f;

// Exponentials are taken in fp32 (v_exp_f32, one step) of the difference to a
// reference value X that the lane has seen, summed over one vector in fp32 and
// beyond that in 64 bits.  X follows the maximum only when that is 16 ahead, so
// nearly never after the first vector.
constexpr int kAhead = 4;   // vectors in flight per lane
constexpr int kKept = 64;   // values kept by a part's second look

// The K best of a part when more than kKept values reach the bound (long runs of
// equal logits): extracted one by one, each from the lane whose next value comes
// first, whose vectors (64 at most, one per lane) are reread.
template <bool BF>
__device__ __noinline__ void part_best_by_one(const BeamParams& p, const char* base, int v0, int v1, float best,
                                              int at, long long out) {
  constexpr int VE = Row<BF>::VE;
  const int lane = threadIdx.x & 63;
  float last_v = INFINITY;
  int last_i = -1;
  for (int r = 0; r < p.K; ++r) {
    const int w = wave_best(best, at);
    const float lv = lane_f(last_v, w);
    const int li = __builtin_amdgcn_readlane(last_i, w);
    const int v = v0 + w + 64 * lane;
    float x[VE];
    if (v < v1)
      Row<BF>::load(base, v * VE, p.V, NAN, x);
    else
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] = NAN;
    // the best of the lane's values that come after (lv, li); NaN never does
    auto after = [&](float av, int ai, float& bv, int& bi) {
      bv = -INFINITY;
      bi = INT_MAX;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const int i = v * VE + j;
        const bool ok = (x[j] < av || (x[j] == av && i > ai)) && (x[j] > bv || bi == INT_MAX);
        bv = ok ? x[j] : bv;
        bi = ok ? i : bi;
      }
    };
    float bv;
    int bi;
    after(lv, li, bv, bi);
    int n = wave_best(bv, bi);
    const float ev = lane_f(bv, n);
    const int ei = __builtin_amdgcn_readlane(bi, n);
    if (lane == 0) {
      p.part_val[out * p.K + r] = ev;
      p.part_idx[out * p.K + r] = ei;
    }
    after(ev, ei, bv, bi);
    n = wave_best(bv, bi);
    const float nv = lane_f(bv, n);
    const int ni = __builtin_amdgcn_readlane(bi, n);
    if (lane == w) {
      best = nv;
      at = ni == INT_MAX ? INT_MAX : ni / VE;
      last_v = ev;
      last_i = ei;
    }
  }
}

template <bool BF>
__global__ void __launch_bounds__(256) beam_rows_kernel(BeamParams p) {
  constexpr int VE = Row<BF>::VE;
  __shared__ float kept_v[4][kKept];
  __shared__ int kept_i[4][kKept];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long job = (long long)blockIdx.x * 4 + wave;
  const int row = (int)(job / p.parts), part = (int)(job % p.parts);
  if (row >= p.B * p.K || p.finished[row]) return;
  const char* base = static_cast<const char*>(p.logits) + (long long)row * p.stride * (BF ? 2 : 4);
  const int nv = (p.V + VE - 1) / VE;
  const int v0 = part * p.vecs, v1 = min(nv, v0 + p.vecs);

  float X = kLowest, best = -INFINITY;
  int at = v0 + lane < v1 ? v0 + lane : INT_MAX;
  double sum = 0.0;
  auto take = [&](int v, const float (&x)[VE]) {
    float mx = x[0];
#pragma unroll
    for (int j = 1; j < VE; ++j) mx = fmaxf(mx, x[j]);
    if (mx > best) {
      best = mx;
      at = v;
      if (mx > X + 16.f) {
        sum *= exp((double)X - (double)mx);
        X = mx;
      }
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      const float d = x[j] - X;
      s += __builtin_amdgcn_exp2f(fmaf(d, kL2eHi, d * kL2eLo));
    }
    sum += (double)s;
  };
  int v = v0 + lane;
  // whole vectors of the row, kAhead at a time
  const int whole = min(v1, p.V / VE);
  for (; v + 64 * (kAhead - 1) < whole; v += 64 * kAhead) {
    typename Row<BF>::Raw u[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) u[a] = Row<BF>::raw(base, (v + 64 * a) * VE);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      float x[VE];
      Row<BF>::split(u[a], x);
      take(v + 64 * a, x);
    }
  }
  for (; v < v1; v += 64) {
    float x[VE];
    Row<BF>::load(base, v * VE, p.V, -INFINITY, x);
    take(v, x);
  }
  // the part's sum: lanes in a fixed order of pairs
  const float Xw = wave_max(X);
  double sw = sum * exp((double)X - (double)Xw);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sw += __shfl_xor(sw, o);
  const long long out = (long long)row * p.parts + part;
  if (lane == 0) {
    p.part_sum[out] = sw;
    p.part_m[out] = Xw;
  }

  // the K lanes whose bests come first, the last of them the bound
  float bound = -INFINITY, hv = best;
  int hi = at, lanes = 0, chosen = 0;
  for (; chosen < p.K; ++chosen) {
    const int w = wave_best(hv, hi);
    if (__builtin_amdgcn_readlane(hi, w) == INT_MAX) {  // fewer lanes than K have values: all of theirs count
      bound = -INFINITY;
      break;
    }
    bound = lane_f(hv, w);
    if (lane == chosen) lanes = w;
    if (lane == w) hv = -INFINITY, hi = INT_MAX;
  }
  // their values that reach it
  const int each = (v1 - v0 + 63) / 64, total = chosen * each;
  int kept = 0;
  for (int t = lane; t - lane < total; t += 64) {
    const int w = __shfl(lanes, min(t / each, chosen - 1));
    const int u = v0 + w + 64 * (t % each);
    const bool in = t < total && u < v1;
    float x[VE];
    if (in)
      Row<BF>::load(base, u * VE, p.V, NAN, x);
    else
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] = NAN;
    float mx = x[0];
#pragma unroll
    for (int j = 1; j < VE; ++j) mx = fmaxf(mx, x[j]);
    if (!__any(mx >= bound)) continue;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      const unsigned long long who = __ballot(x[j] >= bound);
      if (x[j] >= bound) {
        const int pos = kept + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                                         __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
        if (pos < kKept) {
          kept_v[wave][pos] = x[j];
          kept_i[wave][pos] = u * VE + j;
        }
      }
      kept += __popcll(who);
    }
  }
  if (kept > kKept) {
    part_best_by_one<BF>(p, base, v0, v1, best, at, out);
    return;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  float cv = -INFINITY, ov = -INFINITY;
  int ci = INT_MAX, oi = INT_MAX;
  if (lane < kept) {
    cv = kept_v[wave][lane];
    ci = kept_i[wave][lane];
  }
  for (int r = 0; r < p.K; ++r) {
    const int w = wave_best(cv, ci);
    const float ev = lane_f(cv, w);
    const int ei = __builtin_amdgcn_readlane(ci, w);
    if (lane == r) ov = ev, oi = ei;
    if (lane == w) cv = -INFINITY, ci = INT_MAX;
  }
  if (lane < p.K) {
    p.part_val[out * p.K + lane] = ov;
    p.part_idx[out * p.K + lane] = oi;
  }
}

// ---- join ---------------------------------------------------------------------
constexpr int kJoinWaves = 4;

__global__ void __launch_bounds__(kJoinWaves * 64) beam_join_kernel(BeamParams p) {
  __shared__ float heads_v[kJoinWaves][kMaxParts * kMaxK];  // a beam's parts' best
  __shared__ int heads_i[kJoinWaves][kMaxParts * kMaxK];
  __shared__ float val[kMaxK][kMaxK];  // the beams' best, in order
  __shared__ int idx[kMaxK][kMaxK];
  __shared__ double lses[kMaxK], pens[kMaxK];
  __shared__ int parent[kMaxK];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.x / p.copies, copy = blockIdx.x % p.copies;
  const int K = p.K;

  // log-sum-exp and K best of every beam: lane i holds part i's next value
  for (int k = wave; k < K; k += kJoinWaves) {
    const int row = b * K + k;
    const bool fin = p.finished[row] != 0;
    if (lane == 0) pens[k] = pow((5.0 + (p.lengths[row] + (fin ? 0 : 1))) / 6.0, (double)p.alpha);
    if (fin) continue;
    const long long at = (long long)row * p.parts;
    float M = kLowest;
    double s = 0.0;
    if (lane < p.parts) {
      M = p.part_m[at + lane];
      s = p.part_sum[at + lane];
    }
    for (int i = lane; i < p.parts * K; i += 64) {
      heads_v[wave][i] = p.part_val[at * K + i];
      heads_i[wave][i] = p.part_idx[at * K + i];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    const float Mw = wave_max(M);
    s *= exp((double)M - (double)Mw);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
    // no distribution: NaN or +inf among the logits, or all -inf
    if (lane == 0) lses[k] = s > 0.0 && s < INFINITY ? (double)Mw + log(s) : (double)NAN;
    int j = 0, i = INT_MAX;
    float v = -INFINITY;
    if (lane < p.parts) {
      v = heads_v[wave][lane * K];
      i = heads_i[wave][lane * K];
    }
    for (int r = 0; r < K; ++r) {
      const int w = wave_best(v, i);
      if (lane == w) {
        val[k][r] = v;
        idx[k][r] = i;
        const bool more = lane < p.parts && ++j < K;
        v = more ? heads_v[wave][lane * K + j] : -INFINITY;
        i = more ? heads_i[wave][lane * K + j] : INT_MAX;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();

  // the K best of all: lane k holds beam k's next proposal
  if (wave == 0) {
    const bool beam = lane < K;
    const int k = beam ? lane : 0, row = b * K + k;
    const bool fin = p.finished[row] != 0;
    const double score = p.scores[row];
    const int n = p.lengths[row] + (fin ? 0 : 1);
    const double pen = pens[k], lse = fin ? 0.0 : lses[k];
    // proposes rank -inf only
    const bool none = !(score > -INFINITY) || score == INFINITY || isnan(lse);
    int j = 0, tok = 0;
    double cand = -INFINITY, rank = -INFINITY;
    auto next = [&]() {
      if (!beam || j >= K) {
        tok = INT_MAX, cand = rank = -INFINITY;
        return;
      }
      if (none) {
        tok = j, cand = -INFINITY;
      } else if (fin) {
        tok = j == 0 ? p.eos : (j - 1 < p.eos ? j - 1 : j);
        cand = j == 0 ? score : -INFINITY;
      } else {
        tok = idx[k][j];
        cand = score + ((double)val[k][j] - lse);
      }
      rank = cand / pen;
    };
    next();
    for (int r = 0; r < K; ++r) {
      // the largest rank, of equals the lowest beam (its next proposal precedes every other beam's token)
      double br = rank;
      int bk = tok != INT_MAX ? lane : INT_MAX;
#pragma unroll
      for (int o = 1; o < kMaxK; o <<= 1) {
        const double orr = __shfl_xor(br, o);
        const int ok = __shfl_xor(bk, o);
        const bool better = ok != INT_MAX && (bk == INT_MAX || orr > br || (orr == br && ok < bk));
        br = better ? orr : br;
        bk = better ? ok : bk;
      }
      if (lane == bk) {
        parent[r] = lane;
        if (copy == 0) {
          const int o = b * K + r;
          p.tokens[o] = tok;
          p.parents[o] = lane;
          p.scores_out[o] = (float)cand;
          p.finished_out[o] = fin || tok == p.eos;
          p.lengths_out[o] = n;
        }
        ++j;
        next();
      }
    }
  }
  __syncthreads();

  // the chosen beams' states
  const int part = copy * (kJoinWaves * 64) + tid, all = p.copies * (kJoinWaves * 64);
  const long long BK = (long long)p.B * K;
  for (int which = 0; which < 2; ++which) {
    const char* src = which ? p.c : p.h;
    char* dst = which ? p.c_out : p.h_out;
    const int size = which ? 4 : p.h_size;
    if (!src) continue;
    const int unit = p.vec_copy ? 16 : size;
    const int per = p.H * size / unit;  // units of one state row
    const int n = p.L * K * per;
    for (int i = part; i < n; i += all) {
      const int u = i % per, lk = i / per, r = lk % K, l = lk / K;
      const long long to = ((l * BK + (long long)b * K + r) * per + u) * unit;
      const long long from = ((l * BK + (long long)b * K + parent[r]) * per + u) * unit;
      if (unit == 16)
        *reinterpret_cast<uint4*>(dst + to) = *reinterpret_cast<const uint4*>(src + from);
      else if (unit == 4)
        *reinterpret_cast<uint32_t*>(dst + to) = *reinterpret_cast<const uint32_t*>(src + from);
      else
        *reinterpret_cast<uint16_t*>(dst + to) = *reinterpret_cast<const uint16_t*>(src + from);
    }
  }
}

// ---- host ---------------------------------------------------------------------
lstm_status_t check(const lstm_beam_desc_t* d) {
  if (!d) return LSTM_ERR_INVALID_ARG;
  if (d->B < 1 || d->K < 1 || d->V < 1 || d->K > d->V) return LSTM_ERR_INVALID_ARG;
  if (d->dtype != LSTM_F32 && d->dtype != LSTM_BF16) return LSTM_ERR_INVALID_ARG;
  if (d->eos < 0 || d->eos >= d->V || !(d->alpha >= 0.f) || std::isinf(d->alpha)) return LSTM_ERR_INVALID_ARG;
  if (d->L < 0 || d->H < 0 || (d->L == 0) != (d->H == 0)) return LSTM_ERR_INVALID_ARG;
  if (d->logits_stride != 0 && d->logits_stride < d->V) return LSTM_ERR_INVALID_ARG;
  if (d->K > kMaxK || d->V > kMaxV || (long long)d->B * d->K >= 1 << 24) return LSTM_ERR_UNSUPPORTED;
  if ((long long)d->L * d->H * 16 * kMaxK >= 1ll << 31) return LSTM_ERR_UNSUPPORTED;
  return LSTM_OK;
}

// Parts of a row: as many as give every compute unit eight waves, of four
// vectors a lane at least.
void plan(const lstm_beam_desc_t* d, BeamParams* p) {
  const int ve = d->dtype == LSTM_BF16 ? 8 : 4;
  const int nv = (d->V + ve - 1) / ve;
  const long long rows = (long long)d->B * d->K;
  long long n = (2048 + rows - 1) / rows;
  const int most = (nv + 255) / 256;
  if (n > most) n = most;
  const int least = (nv + 64 * kVecsPerLane - 1) / (64 * kVecsPerLane);
  if (n < least) n = least;
  if (n > kMaxParts) n = kMaxParts;
  p->vecs = (int)((nv + n - 1) / n);
  p->parts = (nv + p->vecs - 1) / p->vecs;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" {

size_t lstm_beam_workspace_size(const lstm_beam_desc_t* d) {
  if (check(d) != LSTM_OK) return 0;
  BeamParams p = {};
  plan(d, &p);
  const size_t n = (size_t)d->B * d->K * p.parts;
  return round256(n * 8) + round256(n * 4) + 2 * round256(n * d->K * 4);
}

lstm_status_t lstm_beam_step(const lstm_beam_desc_t* d, const void* logits, const float* scores,
                             const uint8_t* finished, const int32_t* lengths, int32_t* tokens, int32_t* parents,
                             float* scores_out, uint8_t* finished_out, int32_t* lengths_out, const void* h,
                             const float* c, void* h_out, float* c_out, void* ws, hipStream_t stream) {
  const lstm_status_t st = check(d);
  if (st != LSTM_OK) return st;
  if (!logits || !scores || !finished || !lengths || !tokens || !parents || !scores_out || !finished_out ||
      !lengths_out)
    return LSTM_ERR_INVALID_ARG;
  if ((h && !h_out) || (c && !c_out) || ((h || c) && d->L == 0)) return LSTM_ERR_INVALID_ARG;
  const int size = d->dtype == LSTM_BF16 ? 2 : 4;
  if (!aligned(logits, size) || !aligned(h, size) || !aligned(h_out, size)) return LSTM_ERR_INVALID_ARG;
  for (const void* x : {(const void*)scores, (const void*)lengths, (const void*)tokens, (const void*)parents,
                        (const void*)scores_out, (const void*)lengths_out, (const void*)c, (const void*)c_out})
    if (!aligned(x, 4)) return LSTM_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256)) return LSTM_ERR_WORKSPACE;
  BeamParams p = {};
  p.logits = logits, p.scores = scores, p.finished = finished, p.lengths = lengths;
  p.tokens = tokens, p.parents = parents, p.scores_out = scores_out, p.finished_out = finished_out;
  p.lengths_out = lengths_out;
  p.h = (const char*)h, p.c = (const char*)c, p.h_out = (char*)h_out, p.c_out = (char*)c_out;
  p.B = d->B, p.K = d->K, p.V = d->V, p.eos = d->eos, p.L = d->L, p.H = d->H, p.alpha = d->alpha;
  p.h_size = size;
  p.stride = d->logits_stride ? d->logits_stride : d->V;
  plan(d, &p);
  const size_t n = (size_t)d->B * d->K * p.parts;
  char* at = (char*)ws;
  p.part_sum = (double*)at, at += round256(n * 8);
  p.part_m = (float*)at, at += round256(n * 4);
  p.part_val = (float*)at, at += round256(n * d->K * 4);
  p.part_idx = (int*)at;
  p.vec_copy = (d->H * size) % 16 == 0 && (d->H * 4) % 16 == 0 && aligned(h, 16) && aligned(h_out, 16) &&
               aligned(c, 16) && aligned(c_out, 16);
  // about 32 KiB of states a workgroup
  const long long state = (long long)d->L * d->K * d->H * ((h ? size : 0) + (c ? 4 : 0));
  long long copies = state / 32768;
  if (copies < 1) copies = 1;
  if (copies > 64) copies = 64;
  p.copies = (int)copies;

  const long long blocks = ((long long)n + 3) / 4;
  if (d->dtype == LSTM_BF16)
    hipLaunchKernelGGL((beam_rows_kernel<true>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((beam_rows_kernel<false>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  if (hipGetLastError() != hipSuccess) return LSTM_ERR_HIP;
  hipLaunchKernelGGL(beam_join_kernel, dim3((unsigned)(d->B * p.copies)), dim3(256), 0, stream, p);
  return hipGetLastError() == hipSuccess ? LSTM_OK : LSTM_ERR_HIP;
}

}  // extern "C"
