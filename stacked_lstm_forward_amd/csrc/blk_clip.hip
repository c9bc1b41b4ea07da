// The norm of many tensors together, and the tensors scaled to a largest norm.
//
// The tensors are cut into chunks of 4096 elements, and a workgroup has a run of them
// (at most eight workgroups a compute unit), whose tensors it walks over.  Two launches:
// the first leaves every workgroup's sum of squares, the second joins all of them in
// every workgroup, in the same order, and scales.  Bound by memory: two reads and a
// write of every element, the second read backwards, which finds what the first one
// left in the last-level cache: 537 million fp32 values 344 and 816 us (5.5 TB/s for
// both), 131 thousand 3.4 and 4.3 us.
#include "blk_clip.h"

#include "blk_common.h"

namespace lstm {
namespace {

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int n = 1; n < 64; n *= 2) v += __shfl_xor(v, n);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// The entry that holds a chunk: the last one that begins at or before it (empty tensors begin where
// the next one does).
__device__ int entry_of(const ClipEntry* e, int n, long long chunk) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (e[mid].first <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__global__ __launch_bounds__(64) void clip_table_kernel(ClipTableArgs a) {
  for (int i = threadIdx.x; i < a.n; i += 64) a.table[a.at + i] = a.entry[i];
}

__global__ __launch_bounds__(256) void clip_span_kernel(ClipParams p, int2* span) {
  const int g = blockIdx.x * 256 + threadIdx.x;
  if (g >= p.blocks || p.chunks == 0) return;
  span[g] = make_int2(entry_of(p.table, p.n, clip_from(p.chunks, p.blocks, g)),
                      entry_of(p.table, p.n, clip_from(p.chunks, p.blocks, g + 1) - 1));
}

constexpr int kEach = kClipChunk / 256;  // elements of a chunk and thread

// A thread's elements of a chunk: vectors of 16 bytes, one beside another for the threads.
template <bool BF, typename F>
__device__ __forceinline__ void each_vector(int n, F f) {
  constexpr int V = BF ? 8 : 4;
#pragma unroll
  for (int k = 0; k < kEach / V; ++k) {
    const int i = (k * 256 + threadIdx.x) * V;
    if (n == kClipChunk || i < n) f(k, i, n - i < V ? n - i : V);
  }
}

template <bool BF>
__device__ __forceinline__ double squares(const void* src, long long at, int n) {
  typedef typename Dt<BF>::T E;
  constexpr int V = BF ? 8 : 4;
  const E* p = (const E*)src + at;
  Raw<BF, V> r[kEach / V];
#pragma unroll
  for (int k = 0; k < kEach / V; ++k) r[k].clear();
  each_vector<BF>(n, [&](int k, int i, int m) {
    if (m == V)
      r[k].load(p + i);
    else
      r[k].load_part(p + i, m);
  });
  double s = 0;
#pragma unroll
  for (int k = 0; k < kEach / V; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double x = r[k].get(i);
      s = __builtin_fma(x, x, s);
    }
  return s;
}

template <bool BF>
__device__ __forceinline__ void scale(const void* src, void* dst, long long at, int n, double by) {
  typedef typename Dt<BF>::T E;
  constexpr int V = BF ? 8 : 4;
  const E* p = (const E*)src + at;
  E* q = (E*)dst + at;
  Raw<BF, V> r[kEach / V];
  each_vector<BF>(n, [&](int k, int i, int m) {
    if (m == V)
      r[k].load(p + i);
    else
      r[k].load_part(p + i, m);
  });
  each_vector<BF>(n, [&](int k, int i, int m) {
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = (float)(by * r[k].get(j));
    r[k].set(v);
    if (m == V)
      r[k].store_once(q + i);
    else
      r[k].store_part(q + i, m);
  });
}

__device__ __forceinline__ int length_of(const ClipEntry& e, long long chunk) {
  const long long left = e.count - (chunk - e.first) * kClipChunk;
  return left < kClipChunk ? (int)left : kClipChunk;
}

__global__ __launch_bounds__(256) void clip_sum_kernel(ClipParams p) {
  __shared__ double lds[4];
  const long long from = clip_from(p.chunks, p.blocks, blockIdx.x), to = clip_from(p.chunks, p.blocks, blockIdx.x + 1);
  double sum = 0;
  if (from < to) {
    int i = p.span[blockIdx.x].x;
    ClipEntry e = p.table[i];
    for (long long c = from; c < to; ++c) {
      while ((c - e.first) * kClipChunk >= e.count) e = p.table[++i];
      const long long at = (c - e.first) * kClipChunk;
      sum += e.bf16 ? squares<true>(e.src, at, length_of(e, c)) : squares<false>(e.src, at, length_of(e, c));
    }
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) p.part[blockIdx.x] = sum;
}

__global__ __launch_bounds__(256) void clip_scale_kernel(ClipParams p) {
  __shared__ double lds[4];
  const long long from = clip_from(p.chunks, p.blocks, blockIdx.x), to = clip_from(p.chunks, p.blocks, blockIdx.x + 1);
  double sum = 0;
  for (int i = threadIdx.x; i < p.blocks; i += 256) sum += p.part[i];
  const double norm = sqrt(block_sum(sum, lds)), by = norm + p.eps;
  const double c = isinf(p.max_norm) || by == 0. ? 1. : p.max_norm / by;  // (no 0 / 0)
  const double coef = c > 1. ? 1. : c;  // (in 64 bits for the products too: it may be small)
  if (blockIdx.x == 0 && threadIdx.x == 0) p.out[0] = (float)norm, p.out[1] = (float)coef;
  if (from >= to) return;
  int i = p.span[blockIdx.x].y;
  ClipEntry e = p.table[i];
  for (long long k = to - 1; k >= from; --k) {
    while (e.first > k) e = p.table[--i];
    if (!e.dst || (e.dst == e.src && coef == 1.)) continue;
    const long long at = (k - e.first) * kClipChunk;
    if (e.bf16)
      scale<true>(e.src, e.dst, at, length_of(e, k), coef);
    else
      scale<false>(e.src, e.dst, at, length_of(e, k), coef);
  }
}

}  // namespace

hipError_t clip_table_launch(const ClipTableArgs& a, hipStream_t stream) {
  clip_table_kernel<<<1, 64, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t clip_span_launch(const ClipParams& p, int2* span, hipStream_t stream) {
  clip_span_kernel<<<(p.blocks + 255) / 256, 256, 0, stream>>>(p, span);
  return hipGetLastError();
}

hipError_t clip_launch(const ClipParams& p, hipStream_t stream) {
  clip_sum_kernel<<<p.blocks, 256, 0, stream>>>(p);
  clip_scale_kernel<<<p.blocks, 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace lstm
