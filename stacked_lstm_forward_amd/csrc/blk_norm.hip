// Layer norm of a residual sum, and its gradients (formulas: block/lstm_block.h).
//
// A row (one step of one sentence) stays in registers: it is read once, in vectors
// of 16 bytes, 8 or 16 elements a lane, by a group of 4 to 1024 lanes.  Workgroups
// walk over rows, forwards with the next row's loads under way; weight and bias
// stay in registers.  mean and the sum of squares about it take one meeting of the
// group's waves: each wave takes both about its own mean, and the waves' are joined
// by their counts (Chan, Golub and LeVeque, 1979), so nothing cancels; a mean of fp32
// values is corrected by the mean distance to it, which leaves one rounding (0 to 2 %
// of the forward's time).  The gradients' two sums meet the same way; dw and db are summed over a workgroup's
// rows in registers, and the workgroups' sums by a second launch, all in a fixed
// order.
// Bound by memory where rows are many: 8 x 4096 rows of 4096 (bf16, residual) take
// 413 us forwards and backwards with the join, 5.3 TB/s (passes after each other; a
// kernel trace, which parts them, has 198, 218 and 5); by launches, loads and meetings
// after each other where they are few: 16 rows of 4096 5.1 us, 64 x 100 rows of 512
// (fp32) 27 us (12, 13 and 4).
#include "blk_common.h"

namespace lstm {
namespace {

constexpr int kComputeUnits = 256;

template <bool BF>
using Elem = typename Dt<BF>::T;

// What a lane holds of a row: K vectors of V elements, vector k at column (k * TPR + lane) * V.  The vector
// that the row's end cuts is moved back to end with the row: its first `skip` elements are another lane's too,
// count in no sum over the row, and are computed and written alike by both.  (A row has a vector at least:
// shorter ones take V = 1.)
template <bool BF, int E, int TPR, int V>
struct Row {
  static constexpr int K = E / V;
  int col[K], skip[K];  // skip = V: nothing of the row

  __device__ __forceinline__ Row(int lane, int N) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + lane) * V, left = N - c;
      col[k] = left >= V || left <= 0 ? c : N - V;
      skip[k] = left >= V ? 0 : left <= 0 ? V : V - left;
    }
  }
  __device__ __forceinline__ bool has(int k) const { return skip[k] < V; }
  __device__ __forceinline__ bool own(int k, int i) const { return i >= skip[k]; }

  template <bool GBF>
  __device__ __forceinline__ void load(Raw<GBF, V> (&r)[K], const void* base, long long at) const {
    const Elem<GBF>* p = (const Elem<GBF>*)base + at;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (has(k)) r[k].load(p + col[k]);
  }
  // a weight's vector, or the value in its place
  __device__ __forceinline__ void load_one(Raw<BF, V>& r, const void* p, float value, int k) const {
    const float v[8] = {value, value, value, value, value, value, value, value};
    r.set(v);
    if (p && has(k)) r.load((const Elem<BF>*)p + col[k]);
  }
  __device__ __forceinline__ void load_or(Raw<BF, V> (&r)[K], const void* p, float value) const {
#pragma unroll
    for (int k = 0; k < K; ++k) load_one(r[k], p, value, k);
  }
};

// A row's place.
struct At {
  int b, t;
  bool live;  // a row of the launch, and a step of its sentence
};
__device__ __forceinline__ At at_row(const NormParams& p, unsigned row, unsigned rows) {
  const unsigned r = row < rows ? row : 0, b = r / (unsigned)p.T;
  return {(int)b, (int)(r - b * p.T), row < rows && (int)(r - b * p.T) < steps_of(p.lengths, (int)b, p.T)};
}

// This lane's group.  Where it is the wave's, the row's place is worked out in scalar registers.
template <int TPR>
__device__ __forceinline__ int group_of() {
  const int g = threadIdx.x / TPR;
  if constexpr (TPR >= 64) return __builtin_amdgcn_readfirstlane(g);
  return g;
}

// Elements of a wave's (of a group of several) part of a row.
template <int E, int TPR, int V>
__device__ __forceinline__ float wave_count(int wave, int N) {
  int n = 0;
#pragma unroll
  for (int k = 0; k < E / V; ++k) {
    const int left = N - (k * TPR + wave * 64) * V;
    n += left < 0 ? 0 : left > 64 * V ? 64 * V : left;
  }
  return (float)n;
}

constexpr int threads_of(int TPR) { return TPR > 256 ? TPR : 256; }

template <bool BF, int E, int TPR, int V>
__global__ __launch_bounds__(threads_of(TPR)) void norm_fwd_kernel(NormParams p) {
  typedef Row<BF, E, TPR, V> R;
  constexpr int K = R::K, kGroups = threads_of(TPR) / TPR, kWaves = TPR > 64 ? TPR / 64 : 1;  // waves of a group
  constexpr int kLanes = TPR < 64 ? TPR : 64;
  __shared__ float2 part[2][kWaves];
  const int lane = threadIdx.x % TPR, group = group_of<TPR>();
  const unsigned rows = (unsigned)p.B * p.T, step = gridDim.x * kGroups, first = blockIdx.x * kGroups;
  const R at(lane, p.N);

  Raw<BF, V> w[K], bias[K];
  at.load_or(w, p.w, 1.f);
  at.load_or(bias, p.b, 0.f);
  // counts of this lane's wave, and of the wave whose part this lane joins
  const float mine = kWaves > 1 ? wave_count<E, TPR, V>(threadIdx.x / 64, p.N) : p.N;
  const float other = kWaves > 1 ? wave_count<E, TPR, V>(threadIdx.x % kWaves, p.N) : 0.f;
  const float inv = 1.f / p.N;

  Raw<BF, V> x[K], r[K];
  auto fetch = [&](unsigned row) {
    const At a = at_row(p, row, rows);
    if (a.live) {
      at.template load<BF>(x, p.x, a.b * p.sx.b + a.t * p.sx.t);
      if (p.r) at.template load<BF>(r, p.r, a.b * p.sr.b + a.t * p.sr.t);
    }
    return a;
  };
  At next = fetch(first + group);
  int buffer = 0;
  // (the block's rows end together: groups without a row of their own join the meetings)
  for (unsigned lead = first, row = first + group; lead < rows; lead += step, row += step, buffer ^= 1) {
    const At now = next;
    Raw<BF, V> sum[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (p.r) {
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = x[k].get(i) + r[k].get(i);
        sum[k].set(s);
      } else {
        sum[k] = x[k];
      }
      if (!now.live) sum[k].clear();
    }
    next = fetch(row + step);

    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) s1 += at.own(k, i) ? sum[k].get(i) : 0.f;
    float mean = lane_sum<kLanes>(s1);
    mean = mine > 0.f ? mean / mine : 0.f;
    // The long sum's roundings, which may be far more than the values' spread, show in the distances to it.  (Not of
    // bf16 values: where they lie within a factor of 4, the sums of 2^14 of them have 24 bits and are exact; where they
    // do not, the spread is at least 2^-8 of the largest.)
    if constexpr (!BF) {
      float off = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) off += at.own(k, i) ? sum[k].get(i) - mean : 0.f;
      off = lane_sum<kLanes>(off);
      off = mine > 0.f ? off / mine : 0.f;  // (divided: the mean of equal distances is exact, and so that of equal values)
      if (__builtin_fabsf(off) < __builtin_inff()) mean += off;
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = sum[k].get(i) - mean;
        s2 += at.own(k, i) ? d * d : 0.f;
      }
    s2 = lane_sum<kLanes>(s2);
    if constexpr (kWaves > 1) {
      if (threadIdx.x % 64 == 0) part[buffer][threadIdx.x / 64] = make_float2(mean, s2);
      __syncthreads();
      // lane l of every wave joins part l % kWaves: the mean by its distance to the first wave's, which has columns
      const float2 o = part[buffer][threadIdx.x % kWaves];
      const float base = part[buffer][0].x;
      mean = base + lane_sum<kWaves>(other * (o.x - base)) / p.N;
      if (!(__builtin_fabsf(mean) < __builtin_inff())) mean = lane_sum<kWaves>(other * o.x) / p.N;
      const float d = o.x - mean;
      s2 = lane_sum<kWaves>(other * d * d + o.y);
    }
    const float rstd = 1.f / sqrtf(s2 * inv + p.eps);

    if (row < rows) {
      Elem<BF>* y = (Elem<BF>*)p.y + now.b * p.sy.b + now.t * p.sy.t;
      Elem<BF>* z = (Elem<BF>*)p.s + now.b * p.ss.b + now.t * p.ss.t;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!at.has(k)) continue;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
          v[i] = __builtin_fmaf((sum[k].get(i) - mean) * rstd, w[k].get(i), bias[k].get(i));
        Raw<BF, V> out;
        out.set(v);
        if (!now.live) out.clear();
        out.store(y + at.col[k]);
        if (p.s) sum[k].store(z + at.col[k]);
      }
      if (lane == 0) {
        if (p.mean) p.mean[row] = now.live ? mean : 0.f;
        if (p.rstd) p.rstd[row] = now.live ? rstd : 0.f;
      }
    }
  }
}

// dx of every row, and each workgroup's sums of dw and db: part[block][2][N].
template <bool BF, bool GBF, int E, int TPR, int V>
__global__ __launch_bounds__(threads_of(TPR)) void norm_bwd_kernel(NormParams p) {
  typedef Row<BF, E, TPR, V> R;
  constexpr int K = R::K, kGroups = threads_of(TPR) / TPR, kWaves = TPR > 64 ? TPR / 64 : 1;
  constexpr int kLanes = TPR < 64 ? TPR : 64, kCols = E * TPR;
  constexpr bool kLate = kCols > 8192;  // ds and w when they are needed: the registers do not hold them as well
  __shared__ float2 part[2][kWaves];
  __shared__ float total[TPR <= 64 ? kCols : 1];
  const int lane = threadIdx.x % TPR, group = group_of<TPR>();
  const unsigned rows = (unsigned)p.B * p.T, step = gridDim.x * kGroups, first = blockIdx.x * kGroups;
  const R at(lane, p.N);
  const float inv = 1.f / p.N;

  Raw<BF, V> w[K];
  if (!kLate) at.load_or(w, p.w, 1.f);
  float dw[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.f;

  int buffer = 0;
  for (unsigned lead = first, row = first + group; lead < rows; lead += step, row += step, buffer ^= 1) {
    Raw<BF, V> x[K];
    Raw<GBF, V> dy[K], ds[K];
    float mean = 0.f, rstd = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) x[k].clear(), dy[k].clear();
    const At now = at_row(p, row, rows);
    if (now.live) {
      at.template load<BF>(x, p.x, now.b * p.ss.b + now.t * p.ss.t);
      at.template load<GBF>(dy, p.dy, now.b * p.sdy.b + now.t * p.sdy.t);
      if (p.ds && !kLate) at.template load<GBF>(ds, p.ds, now.b * p.sds.b + now.t * p.sds.t);
      mean = p.mean[row], rstd = p.rstd[row];
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (kLate) {
        __builtin_amdgcn_sched_barrier(0);
        at.load_one(w[k], p.w, 1.f, k);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = k * V + i;
        const float n = (x[k].get(i) - mean) * rstd, g0 = dy[k].get(i), g = at.own(k, i) ? g0 * w[k].get(i) : 0.f;
        dw[e] += g0 * n;
        db[e] += g0;
        s1 += g;
        s2 += g * n;
      }
    }
    // n and g are made again below from what was loaded: registers for them cost waves
#pragma unroll
    for (int k = 0; k < K; ++k) x[k].hide(), dy[k].hide();
    s1 = lane_sum<kLanes>(s1);
    s2 = lane_sum<kLanes>(s2);
    if constexpr (kWaves > 1) {
      if (threadIdx.x % 64 == 0) part[buffer][threadIdx.x / 64] = make_float2(s1, s2);
      __syncthreads();
      const float2 o = part[buffer][threadIdx.x % kWaves];
      s1 = lane_sum<kWaves>(o.x);
      s2 = lane_sum<kWaves>(o.y);
    }
    s1 *= inv, s2 *= inv;
    if (row < rows) {
      Elem<GBF>* q = (Elem<GBF>*)p.dx + now.b * p.sdx.b + now.t * p.sdx.t;
      const Elem<GBF>* z = (const Elem<GBF>*)p.ds + now.b * p.sds.b + now.t * p.sds.t;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!at.has(k)) continue;
        if (kLate) {
          if (p.ds && now.live) ds[k].load(z + at.col[k]);
          at.load_one(w[k], p.w, 1.f, k);
        }
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float n = (x[k].get(i) - mean) * rstd, g = dy[k].get(i) * w[k].get(i);
          d[i] = (g - s1 - n * s2) * rstd;
          if (p.ds) d[i] += ds[k].get(i);
        }
        Raw<GBF, V> out;
        out.set(d);
        if (!now.live) out.clear();
        out.store(q + at.col[k]);
        if (kLate) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* acc = which ? db : dw;
    // (the only workgroup's sums are the results)
    float* to = p.blocks > 1 ? p.part + ((long long)blockIdx.x * 2 + which) * p.N : which ? p.db : p.dw;
    // the wave's groups
#pragma unroll
    for (int n = TPR; n < 64; n *= 2)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += __shfl_xor(acc[e], n);
    if constexpr (TPR <= 64) {
      // the waves, one after the other
      for (int o = 0; o < 4; ++o) {
        __syncthreads();
        if ((int)threadIdx.x / 64 == o && (int)threadIdx.x % 64 < TPR)
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (at.has(e / V)) {
              float& t = total[((e / V) * TPR + lane) * V + e % V];
              t = o ? t + acc[e] : acc[e];
            }
      }
      __syncthreads();
    }
    if (to && (TPR > 64 || threadIdx.x < TPR))
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!at.has(k)) continue;
        Raw<false, V> out;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = TPR <= 64 ? total[(k * TPR + lane) * V + i] : acc[k * V + i];
        out.set(v);
        out.store(to + at.col[k]);
      }
  }
}

// dw and db: 32 columns of part [blocks][2 N] a workgroup, each of 32 groups of lanes every 32nd row.
__global__ __launch_bounds__(1024) void norm_join_kernel(NormParams p) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x % 32, group = threadIdx.x / 32, cols = 2 * p.N;
  const int c = blockIdx.x * 32 + lane;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < cols)
    for (int i = group; i < p.blocks; i += 256) {
      float v[8];  // (all loads of a round are under way before the first is used)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p.part[(long long)(i + 32 * j < p.blocks ? i + 32 * j : i) * cols + c];
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += i + 32 * j < p.blocks ? v[j] : 0.f;
    }
  sums[group][lane] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
  // lane l of group g: row l of column g, summed over 32 lanes
  const float v = lane_sum<32>(sums[lane][group]);
  const int to = blockIdx.x * 32 + group;
  if (lane || to >= cols) return;
  if (to < p.N) {
    if (p.dw) p.dw[to] = v;
  } else if (p.db) {
    p.db[to - p.N] = v;
  }
}

// Lanes a row and elements a lane: the fewest lanes, since groups within a wave need no
// meeting and one wave's groups no barrier.
struct Shape {
  int tpr, e;
};
Shape shape_of(int N) {
  if (N < 8) return {4, 2};  // one element at a time
  if (N <= 32) return {4, 8};
  if (N <= 64) return {8, 8};
  if (N <= 128) return {16, 8};
  if (N <= 512) return {64, 8};
  if (N <= 1024) return {64, 16};
  if (N <= 2048) return {256, 8};
  if (N <= 4096) return {256, 16};
  if (N <= 8192) return {1024, 8};
  return {1024, 16};
}

// Workgroups: as many as the compute units hold at once, and each with as many rows to walk over, at
// least `least` for a group of lanes.
int blocks_of(const NormParams& p, int per_unit, int least) {
  const Shape s = shape_of(p.N);
  const int groups = threads_of(s.tpr) / s.tpr;
  const long long n = ((long long)p.B * p.T + groups - 1) / groups, most = kComputeUnits * per_unit;
  long long walk = (n + most - 1) / most;
  if (walk < least) walk = least;
  return (int)((n + walk - 1) / walk);
}
// About what the registers let a compute unit hold (with 8 elements a lane six to eight, with 16 five of bf16 and
// four of fp32, whose fifth follows the others: 8 x 4096 rows of 4096, fp32, 427 us, 5.0 TB/s), and backwards less:
// each leaves 2 N sums behind (8 x 4096 rows of 4096: 237 us with four workgroups a compute unit, 222 with three, 204
// with two, 270 with one).
int fwd_blocks(const NormParams& p) {
  const Shape s = shape_of(p.N);
  return blocks_of(p, s.tpr > 256 ? 1 : s.e == 8 ? 6 : 5, 1);
}
int bwd_blocks(const NormParams& p) {
  const Shape s = shape_of(p.N);
  return blocks_of(p, s.tpr > 256 ? 1 : s.tpr < 64 ? 5 : s.e == 8 ? 3 : 2, 4);
}

template <bool BF, int E, int TPR>
void fwd(const NormParams& p, hipStream_t stream) {
  norm_fwd_kernel<BF, E, TPR, E == 2 ? 1 : BF ? 8 : 4><<<fwd_blocks(p), threads_of(TPR), 0, stream>>>(p);
}
template <bool BF, bool GBF, int E, int TPR>
void bwd(const NormParams& p, hipStream_t stream) {
  norm_bwd_kernel<BF, GBF, E, TPR, E == 2 ? 1 : BF ? 8 : 4><<<p.blocks, threads_of(TPR), 0, stream>>>(p);
}

#define NORM_SHAPES(call)                                  \
  switch (s.tpr * 32 + s.e) {                              \
    case 4 * 32 + 2: call(2, 4); break;                    \
    case 4 * 32 + 8: call(8, 4); break;                    \
    case 8 * 32 + 8: call(8, 8); break;                    \
    case 16 * 32 + 8: call(8, 16); break;                  \
    case 64 * 32 + 8: call(8, 64); break;                  \
    case 64 * 32 + 16: call(16, 64); break;                \
    case 256 * 32 + 8: call(8, 256); break;                \
    case 256 * 32 + 16: call(16, 256); break;              \
    case 1024 * 32 + 8: call(8, 1024); break;              \
    default: call(16, 1024);                               \
  }

}  // namespace

size_t norm_bwd_parts(const NormParams& p) { return (size_t)bwd_blocks(p) * 2 * p.N; }

hipError_t norm_fwd_launch(const NormParams& p, bool bf16, hipStream_t stream) {
  const Shape s = shape_of(p.N);
#define CALL(E, TPR) bf16 ? fwd<true, E, TPR>(p, stream) : fwd<false, E, TPR>(p, stream)
  NORM_SHAPES(CALL)
#undef CALL
  return hipGetLastError();
}

hipError_t norm_bwd_launch(const NormParams& params, bool bf16, bool grad_bf16, hipStream_t stream) {
  NormParams p = params;
  const Shape s = shape_of(p.N);
  p.blocks = bwd_blocks(p);
  if (!p.dw && !p.db) p.part = nullptr;
#define CALL(E, TPR)                                                            \
  !bf16 ? bwd<false, false, E, TPR>(p, stream)                                  \
        : grad_bf16 ? bwd<true, true, E, TPR>(p, stream) : bwd<true, false, E, TPR>(p, stream)
  NORM_SHAPES(CALL)
#undef CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.part || p.blocks == 1) return e;
  norm_join_kernel<<<(2 * p.N + 31) / 32, 1024, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace lstm
