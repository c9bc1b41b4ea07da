// One step of beam search (include/decoder/lstm_dec.h): two or three launches.
//
//   rows     one wave per part of a beam's row of logits reads it once, in steps of
//            64 vectors of 16 bytes: it sums the exponentials and collects the
//            values above a bound that K values of earlier steps reach (at first
//            the K best lanes of the first steps), and raises the bound whenever
//            its list is full.  A part whose list overflows by itself (long runs
//            of equal or rising logits) or holds fewer than K finite values is
//            read again and its K best are extracted one by one.
//   join     one sentence per workgroup: a wave per beam takes its log-sum-exp in
//            64 bits and its K best from its parts; then each of the K*K proposals
//            counts those that precede it.
//   states   a wave per state row copies the chosen beams' states (where they are
//            few, the join does).
//
// The order of every sum and every comparison is by index in the row, never by
// address: beams with equal rows get equal sums, and their ties stay ties.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <climits>
#include <cmath>

#include "decoder/lstm_dec.h"  // include/ is on the include path
#include "dec_grid.h"
#include "lstm_common.h"

namespace lstm {
namespace {

constexpr int kMaxK = 16;
constexpr int kMaxParts = 64;
constexpr int kVecsPerLane = 64;  // of one part: an extraction rereads one lane's with one load
constexpr int kCopyBytes = 16384; // states of a sentence that the join copies
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
  int copy;              // the join copies the states
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

constexpr double kLog2e = 1.44269504088896340736;
constexpr float kL2e = (float)kLog2e;
constexpr double kTail = 1.0 - (double)kL2e / kLog2e;  // what the rounded factor takes from an exponent
constexpr float kLowest = -3.402823466e38f;
constexpr int kAhead = 4;   // steps in flight
constexpr int kList = 64;   // values collected before the bound is raised: one a lane

// The K best of a part, extracted one by one: each from the lane whose next value
// comes first in the order (value falling, index rising), whose vectors (64 at
// most, one per lane) are reread.
template <bool BF>
__device__ __forceinline__ void part_best_by_one(const BeamParams& p, const char* base, int v0, int v1, int lane,
                                                 long long out) {
  constexpr int VE = Row<BF>::VE;
  float best = -INFINITY, last_v = INFINITY;
  int at = v0 + lane < v1 ? v0 + lane : INT_MAX, last_i = -1;
  for (int v = v0 + lane; v < v1; v += 64) {
    float x[VE];
    Row<BF>::load(base, v * VE, p.V, -INFINITY, x);
    float mx = x[0];
#pragma unroll
    for (int j = 1; j < VE; ++j) mx = fmaxf(mx, x[j]);
    if (mx > best) best = mx, at = v;
  }
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

// A wave's own LDS accesses take effect in order; only the compiler has to keep them so.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

// The K best of a wave's list of n (at most 64), in order, to its front and to lanes 0 .. K-1.
// `cv` is what is left of the list: a value a lane, -inf where there is none.
__device__ __forceinline__ void list_best(float* lv, int* li, int n, int K, int lane, float& ov, int& oi, float& cv) {
  wave_lds_fence();
  cv = -INFINITY;
  int ci = INT_MAX;
  if (lane < n) cv = lv[lane], ci = li[lane];
  ov = -INFINITY, oi = INT_MAX;
  for (int r = 0; r < K; ++r) {
    const int w = wave_best(cv, ci);
    const float ev = lane_f(cv, w);
    const int ei = __builtin_amdgcn_readlane(ci, w);
    if (lane == r) ov = ev, oi = ei;
    if (lane == w) cv = -INFINITY, ci = INT_MAX;
  }
  wave_lds_fence();
  if (lane < K) lv[lane] = ov, li[lane] = oi;
  wave_lds_fence();
}

// The sum.  Values that enter the list are the largest so far; their exponentials
// are taken in 64 bits when they leave it.  The others' are taken in fp32
// (v_exp_f32, one step) of one fused product x * a - M, M the rounded a * X for a
// reference X at most 1 below the largest value: exact before its one rounding, so
// that the error is relative to the difference from X.  They are summed over one
// vector in fp32 and beyond that in 64 bits.  M's own rounding and the first-order
// effect of a's (kTail times the sum's mean difference from X, a vector's maximum
// standing for its values) are taken out of the sum at its end.  Together within
// 2^-19 of the sum if every rounding of the fp32 part went the same way, in which
// case the proposals of beams closer than that could change places; normal logits of
// deviation 0.5 to 5 leave 2^-26 (1000 values) to 2^-29 (131072); where the listed
// values hold nearly all of the sum, it is as exact as 64 bits.  All exponentials in
// fp32, with X up to 16 below the largest value, left up to 2^-20 (the step below:
// 152 us, now 154).  The exponentials are taken before a step's list is looked at: after
// it (154 and 167 us), or of values changed by it (205), they wait for it.
//
// 2048 rows of 131072 bf16 values, 85 % of them read: 121 us, 3.8 TB/s; vector
// instructions take 71 % of that time (eight exponentials at a quarter of the
// rate per vector, and the list).  320 rows of 32007: 15 us, latency: a wave has
// nine steps, and its list to sort.  Keeping vectors instead of values in the list
// (18.9 and 129 us, then 15 and 124), or a first bound from maxima of groups of lanes
// (17.3 and 131: more to collect), was slower; rereading the best lanes' vectors at the
// end instead of a list 19 and 183.
template <bool BF>
__global__ void __launch_bounds__(256) beam_rows_kernel(BeamParams p) {
  constexpr int VE = Row<BF>::VE;
  typedef typename Row<BF>::Raw Raw;
  __shared__ float list_v[4][kList];
  __shared__ int list_i[4][kList];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long job = (long long)blockIdx.x * 4 + wave;
  const int row = (int)(job / p.parts), part = (int)(job % p.parts);
  if (row >= p.B * p.K) return;
  const char* base = static_cast<const char*>(p.logits) + (long long)row * p.stride * (BF ? 2 : 4);
  const int nv = (p.V + VE - 1) / VE;
  const int v0 = part * p.vecs, v1 = min(nv, v0 + p.vecs);
  float* lv = list_v[wave];
  int* li = list_i[wave];

  // kAhead steps from vector s on: the reads, and a step's values, past the part or
  // the row -inf
  const int whole = min(v1, p.V / VE);
  auto fetch = [&](int s, Raw (&u)[kAhead]) {
    if (whole <= v0) return;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) u[a] = Row<BF>::raw(base, min(s + lane + 64 * a, whole - 1) * VE);
  };
  auto values = [&](const Raw& u, int s, int a, float (&x)[VE]) {
    Row<BF>::split(u, x);
    const int v = s + lane + 64 * a;
    if (s + 64 * (a + 1) > whole && v >= whole) {
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] = -INFINITY;
      if (v < v1) Row<BF>::load(base, v * VE, p.V, -INFINITY, x);
    }
  };
  auto max_of = [&](const float (&x)[VE]) {
    float mx = x[0];
#pragma unroll
    for (int j = 1; j < VE; ++j) mx = fmaxf(mx, x[j]);
    return mx;
  };

  // the first steps: the reference and the first bound
  Raw u0[kAhead] = {}, u1[kAhead] = {};
  fetch(v0, u0);
  if (p.finished[row]) return;  // read beside the first steps
  if (v0 + 64 * kAhead < v1) fetch(v0 + 64 * kAhead, u1);
  float first[kAhead][VE];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) values(u0[a], v0, a, first[a]);
  float hv = max_of(first[0]);
#pragma unroll
  for (int a = 1; a < kAhead; ++a) hv = fmaxf(hv, max_of(first[a]));
  float X = fmaxf(wave_max(hv), kLowest), bound = -INFINITY;
  for (int r = 0; r < p.K; ++r) {
    const int w = wave_best(hv, lane);
    bound = lane_f(hv, w);
    if (lane == w) hv = -INFINITY;
  }
  // where a * X could overflow, differences are 0 or beyond any exponent
  auto by = [](float X) { return fabsf(X) < 1e37f ? kL2e : 1.f; };
  float coef = by(X), M = coef * X;

  double sum = 0.0, exact = 0.0;  // in units of 2^M, and of exp(X)
  float tilt = 0.f;               // sum of exponentials times their vectors' differences from X
  int kept = 0;
  bool full = false;
  // a step's values of at least `least`, and of at least the bound where that has
  // been raised within the step: later values of its size come after the K that
  // reached it.  Their exponentials become 0.
  auto collect = [&](const float (&x)[VE], int v, float least, float (&e)[VE]) {
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      unsigned long long who = __ballot(x[j] >= least);
      if (who == 0 || full) continue;
      if (kept + __popcll(who) > kList) {
        float ov, rest;
        int oi;
        list_best(lv, li, kept, p.K, lane, ov, oi, rest);
        sum += (double)__builtin_amdgcn_exp2f(fmaf(rest, coef, -M));
        if (kept >= p.K) least = bound = fmaxf(bound, lane_f(ov, p.K - 1));
        kept = min(kept, p.K);
        who = __ballot(x[j] >= least);
        full = kept + __popcll(who) > kList;
        if (full) continue;
      }
      e[j] = x[j] >= least ? 0.f : e[j];
      if (x[j] >= least) {
        const int pos = kept + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                                         __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
        lv[pos] = x[j];
        li[pos] = v * VE + j;
      }
      kept += __popcll(who);
    }
  };
  auto exponentials = [&](const float (&x)[VE], float (&e)[VE]) {
#pragma unroll
    for (int j = 0; j < VE; ++j) e[j] = __builtin_amdgcn_exp2f(fmaf(x[j], coef, -M));
  };
  auto add = [&](const float (&e)[VE], float mx) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VE; ++j) s += e[j];
    sum += (double)s;
    tilt = fmaf(s, fmaxf(mx - X, -128.f), tilt);  // (s is 0 before that)
  };
  // the fp32 part in units of exp(X)
  auto settled = [&]() { return (sum + kTail * (double)tilt) * exp2((double)M - (double)coef * (double)X); };
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    const float least = fmaxf(bound, kLowest);
    const float mx = max_of(first[a]);
    float e[VE];
    exponentials(first[a], e);
    if (__any(mx >= least)) collect(first[a], v0 + lane + 64 * a, least, e);
    add(e, mx);
  }
  auto take = [&](const float (&x)[VE], int v) {
    const float mx = max_of(x);
    float e[VE];
    exponentials(x, e);
    if (__any(mx > bound)) {
      if (__any(mx > X + 1.f)) {
        const float top = wave_max(mx);
        exact = (exact + settled()) * exp((double)X - (double)top);
        sum = 0.0;
        tilt = 0.f;
        X = top;
        coef = by(X);
        M = coef * X;
        exponentials(x, e);
      }
      // the least value above the bound
      const int bits = __builtin_bit_cast(int, bound);
      const float least = bound < kLowest ? kLowest
                          : bound == 0.f  ? __builtin_bit_cast(float, 1)
                                          : __builtin_bit_cast(float, bound > 0.f ? bits + 1 : bits - 1);
      collect(x, v, least, e);
    }
    add(e, mx);
  };
  auto batch = [&](const Raw (&u)[kAhead], int s) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      float x[VE];
      values(u[a], s, a, x);
      take(x, s + lane + 64 * a);
    }
  };
  for (int s = v0 + 64 * kAhead; s < v1; s += 128 * kAhead) {
    if (s + 64 * kAhead < v1) fetch(s + 64 * kAhead, u0);
    batch(u1, s);
    if (s + 64 * kAhead >= v1) break;
    if (s + 128 * kAhead < v1) fetch(s + 128 * kAhead, u1);
    batch(u0, s + 64 * kAhead);
  }
  wave_lds_fence();
  if (lane < kept) exact += exp((double)lv[lane] - (double)X);
  exact += settled();

  // the part's sum: lanes in a fixed order of pairs
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) exact += __shfl_xor(exact, o);
  const long long out = (long long)row * p.parts + part;
  if (lane == 0) {
    p.part_sum[out] = exact;
    p.part_m[out] = X;
  }
  if (full || kept < p.K) {
    part_best_by_one<BF>(p, base, v0, v1, lane, out);
    return;
  }
  float ov, rest;
  int oi;
  list_best(lv, li, kept, p.K, lane, ov, oi, rest);
  if (lane < p.K) {
    p.part_val[out * p.K + lane] = ov;
    p.part_idx[out * p.K + lane] = oi;
  }
}

// ---- join ---------------------------------------------------------------------
// Row i of layer l of the states to row `from` of the sources, by n threads.
__device__ __forceinline__ void copy_row(const BeamParams& p, int which, long long from, long long to, int at, int n) {
  const int size = which ? 4 : p.h_size, bytes = p.H * size;
  const char* src = (which ? p.c : p.h) + from * bytes;
  char* dst = (which ? p.c_out : p.h_out) + to * bytes;
  if (p.vec_copy) {
    const int per = bytes / 16;
    const u32x4_a4* from4 = reinterpret_cast<const u32x4_a4*>(src);
    for (int i = at; i < per; i += 4 * n) {
      u32x4_a4 x[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) x[a] = from4[min(i + a * n, per - 1)];
#pragma unroll
      for (int a = 0; a < 4; ++a)
        if (i + a * n < per) reinterpret_cast<u32x4_a4*>(dst)[i + a * n] = x[a];
    }
  } else if (size == 4) {
    for (int i = at; i < p.H; i += n) reinterpret_cast<uint32_t*>(dst)[i] = reinterpret_cast<const uint32_t*>(src)[i];
  } else {
    for (int i = at; i < p.H; i += n) reinterpret_cast<uint16_t*>(dst)[i] = reinterpret_cast<const uint16_t*>(src)[i];
  }
}

// A wave per beam.  Latency: 5.5 us for one sentence of 4 beams of 8 parts, 9 us for
// 256 sentences of 8 beams.
__global__ void __launch_bounds__(kMaxK * 64) beam_join_kernel(BeamParams p) {
  extern __shared__ char heads[];  // [K][parts * K] values, then indexes: a beam's parts' best
  __shared__ double rank[kMaxK * kMaxK], cand[kMaxK * kMaxK];  // the beams' proposals, in order
  __shared__ int tok[kMaxK * kMaxK];
  __shared__ int parent[kMaxK];
  const int tid = threadIdx.x, lane = tid & 63, k = tid >> 6;
  const int b = blockIdx.x, K = p.K, row = b * K + k, n = p.parts * K;
  float* hv = reinterpret_cast<float*>(heads) + k * n;
  int* hi = reinterpret_cast<int*>(heads) + (K + k) * n;

  // log-sum-exp and K best of the beam: lane i holds part i's next value
  const bool fin = p.finished[row] != 0;
  const double score = p.scores[row];
  const int length = p.lengths[row] + (fin ? 0 : 1);
  float M = kLowest;
  double s = 0.0;
  if (!fin) {
    const long long at = (long long)row * p.parts;
    if (lane < p.parts) {
      M = p.part_m[at + lane];
      s = p.part_sum[at + lane];
    }
    for (int i = lane; i < n; i += 64) {
      hv[i] = p.part_val[at * K + i];
      hi[i] = p.part_idx[at * K + i];
    }
  }
  const double pen = p.alpha == 0.f ? 1.0 : pow((5.0 + length) / 6.0, (double)p.alpha);
  wave_lds_fence();
  float ov = -INFINITY;  // lane r: the beam's r-th best
  int oi = INT_MAX;
  double lse = 0.0;
  if (!fin) {
    const float Mw = wave_max(M);
    s *= exp((double)M - (double)Mw);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
    // no distribution: NaN or +inf among the logits, or all -inf
    // (one lane's: the compiler may fuse a lane's own product into its sum, and
    // equal logits must give equal ranks)
    lse = __shfl(s > 0.0 && s < INFINITY ? (double)Mw + log(s) : (double)NAN, 0);
    int j = 0, i = INT_MAX;
    float v = -INFINITY;
    if (lane < p.parts) v = hv[lane * K], i = hi[lane * K];
    for (int r = 0; r < K; ++r) {
      const int w = wave_best(v, i);
      const float ev = lane_f(v, w);
      const int ei = __builtin_amdgcn_readlane(i, w);
      if (r == 0 && lse < ev) lse = ev;  // no probability above 1
      if (lane == r) ov = ev, oi = ei;
      if (lane == w) {
        const bool more = lane < p.parts && ++j < K;
        v = more ? hv[lane * K + j] : -INFINITY;
        i = more ? hi[lane * K + j] : INT_MAX;
      }
    }
  }
  if (lane < K) {
    // proposes rank -inf only
    const bool none = !(score > -INFINITY) || score == INFINITY || isnan(lse);
    int t;
    double c = -INFINITY;
    if (none) {
      t = lane;
    } else if (fin) {
      t = lane == 0 ? p.eos : (lane - 1 < p.eos ? lane - 1 : lane);
      if (lane == 0) c = score;
    } else {
      t = oi;
      c = score + ((double)ov - lse);
    }
    const double r = c / pen;
    tok[k * K + lane] = t;
    cand[k * K + lane] = c;
    rank[k * K + lane] = isnan(r) ? -INFINITY : r;
  }
  __syncthreads();

  // Each proposal's place is the number of those before it: of a larger rank, or
  // of an equal one from a lower beam or, in its own beam, further ahead.
  if (tid < K * K) {
    const double r = rank[tid];
    int place = 0;
    for (int i = 0; i < K * K; ++i) place += rank[i] > r || (rank[i] == r && i < tid);
    if (place < K) {
      const int from = tid / K, o = b * K + place;
      const bool f = p.finished[b * K + from] != 0;
      parent[place] = from;
      p.tokens[o] = tok[tid];
      p.parents[o] = from;
      p.scores_out[o] = (float)cand[tid];
      p.finished_out[o] = f || tok[tid] == p.eos;
      p.lengths_out[o] = p.lengths[b * K + from] + (f ? 0 : 1);
    }
  }
  if (!p.copy) return;
  __syncthreads();
  const long long BK = (long long)p.B * K;
  for (int l = 0; l < p.L; ++l) {
    if (p.h) copy_row(p, 0, l * BK + (long long)b * K + parent[k], l * BK + row, lane, 64);
    if (p.c) copy_row(p, 1, l * BK + (long long)b * K + parent[k], l * BK + row, lane, 64);
  }
}

// A wave per row of h and of c: 16384 rows of 3 or 6 KiB read and written in 23 us,
// 6.6 TB/s (in the join's workgroups, each with a join of its own, 65).
__global__ void __launch_bounds__(256) beam_states_kernel(BeamParams p) {
  const long long BK = (long long)p.B * p.K, job = (long long)grid_block() * 4 + (threadIdx.x >> 6);
  const int which = p.h ? (p.c ? (int)(job & 1) : 0) : 1;
  const long long at = p.h && p.c ? job >> 1 : job;
  if (at >= p.L * BK) return;
  const long long l = at / BK, r = at % BK;
  copy_row(p, which, l * BK + r / p.K * p.K + p.parents[r], at, threadIdx.x & 63, 64);
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
  if ((long long)d->L * d->H * 16 * kMaxK >= 1ll << 31 || (long long)d->B * d->K * d->L >= 1ll << 31)
    return LSTM_ERR_UNSUPPORTED;
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
  const long long state = (long long)d->L * d->K * d->H * ((h ? size : 0) + (c ? 4 : 0));
  p.copy = state > 0 && state <= kCopyBytes;

  const long long blocks = ((long long)n + 3) / 4;
  if (d->dtype == LSTM_BF16)
    hipLaunchKernelGGL((beam_rows_kernel<true>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((beam_rows_kernel<false>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  if (hipGetLastError() != hipSuccess) return LSTM_ERR_HIP;
  hipLaunchKernelGGL(beam_join_kernel, dim3((unsigned)d->B), dim3(d->K * 64), (size_t)p.parts * d->K * d->K * 8, stream,
                     p);
  if (hipGetLastError() != hipSuccess) return LSTM_ERR_HIP;
  if (state > kCopyBytes) {
    const long long jobs = (long long)d->L * d->B * d->K * ((h ? 1 : 0) + (c ? 1 : 0));
    hipLaunchKernelGGL(beam_states_kernel, grid_of((jobs + 3) / 4), dim3(256), 0, stream, p);
    if (hipGetLastError() != hipSuccess) return LSTM_ERR_HIP;
  }
  return LSTM_OK;
}

}  // extern "C"
