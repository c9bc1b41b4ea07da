// Attention over encoder outputs: joining the parts of a split key axis, and
// the row statistics of the backward pass.
#include "dec_attn.h"
#include "dec_attn_launch.h"

namespace lstm {
namespace {

// Bound by the reading of the parts: 25600 rows of two parts of 80, 8.5 us (9.2 with
// what the rounding leaves).
// LR lanes (a power of two, 4 columns each) join one row's parts: with m the
// parts' largest maximum, o = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i.
template <typename T, int LR>
__global__ void __launch_bounds__(256) attn_combine_kernel(AttnParams p) {
  const long long row = (long long)blockIdx.x * (256 / LR) + threadIdx.x / LR;
  const int c = (threadIdx.x % LR) * 4;
  if (row >= (long long)p.B * p.Hkv * p.rows) return;
  const float* ml = p.part_ml + row * p.nsplit * 2;
  float m = -INFINITY;
  for (int i = 0; i < p.nsplit; ++i) m = fmaxf(m, ml[2 * i]);
  const float mu = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  const float* po = p.part_o + row * p.nsplit * p.D + c;
  for (int i = 0; i < p.nsplit; ++i) {
    const float w = exp2_fast(ml[2 * i] - mu);
    l += w * ml[2 * i + 1];
    if (c < p.D) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(po + (long long)i * p.D);
      o += x * w;
    }
  }
  const int r = (int)(row % p.rows);
  const long long bh = row / p.rows;
  const int b = (int)(bh / p.Hkv), t = r / p.G, hq = (int)(bh % p.Hkv) * p.G + r % p.G;
  if (c < p.D) {
    o *= l == 0.f ? 0.f : 1.f / l;
    char* at = p.o + b * p.so.b + t * p.so.t + hq * p.so.h + c * AT<T>::SZ;
    if constexpr (AT<T>::BF) {
      const uint2 u = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
      *reinterpret_cast<uint2*>(at) = u;
      if (p.o_rest)
        *reinterpret_cast<uint2*>(p.o_rest + (row * p.D + c) * 2) =
            make_uint2(rest_bf16(o[0], o[1], u.x), rest_bf16(o[2], o[3], u.y));
    } else {
      *reinterpret_cast<f32x4*>(at) = o;
    }
  }
  if (c == 0 && p.lse) p.lse[((long long)b * p.Hq + hq) * p.Tq + t] = mu * kLn2 + logf(l);
}

template <typename T>
hipError_t combine(const AttnParams& p, hipStream_t s) {
  const long long rows = (long long)p.B * p.Hkv * p.rows;
  auto go = [&](auto kernel, int lr) {
    const long long n = (rows + 256 / lr - 1) / (256 / lr);  // few: a split has less than 256 row tiles
    hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(256), 0, s, p);
    return hipGetLastError();
  };
  if (p.D <= 32) return go(attn_combine_kernel<T, 8>, 8);
  if (p.D <= 64) return go(attn_combine_kernel<T, 16>, 16);
  if (p.D <= 128) return go(attn_combine_kernel<T, 32>, 32);
  return go(attn_combine_kernel<T, 64>, 64);
}

// Row statistics of the backward pass, in the order of the row list: -lse in
// base-2 units (-inf where the row has no key) and -delta = -<dout, o>, o with what
// its rounding to bf16 left where the forward kept that: without it delta's error
// reaches all of a row's dz (2-norm errors of dq against 64 bits 0.0018 to 0.0020
// instead of 0.0017 for 10 to 200 keys, more where one key decides).  16 lanes a row.
// Bound by the reading of o, its rest and dout: 98304 rows of 128 bf16 values, 14.0 us
// = 5.4 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) attn_stats_kernel(AttnParams p) {
  constexpr int SZ = AT<T>::SZ;
  const long long row = (long long)grid_block() * 16 + threadIdx.x / 16;
  if (row >= (long long)p.B * p.Hkv * p.rows) return;
  const int r = (int)(row % p.rows), bh = (int)(row / p.rows);
  const int b = bh / p.Hkv, t = r / p.G, h = (bh % p.Hkv) * p.G + r % p.G;
  const char* o = p.o_in + b * p.so.b + t * p.so.t + h * p.so.h;
  const char* d = p.dout + b * p.sdo.b + t * p.sdo.t + h * p.sdo.h;
  float sum = 0.f;
  const char* rest = p.o_rest + row * p.D * 2;
  for (int c = (threadIdx.x & 15) * 16; c < p.D * SZ; c += 256) {
    const uint4 x = *reinterpret_cast<const uint4*>(o + c), y = *reinterpret_cast<const uint4*>(d + c);
    uint4 z = make_uint4(0, 0, 0, 0);
    if (AT<T>::BF && p.o_rest) z = *reinterpret_cast<const uint4*>(rest + c);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w}, zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (AT<T>::BF) {
        sum = fmaf(bf16_lo(xs[j]) + bf16_lo(zs[j]), bf16_lo(ys[j]), sum);
        sum = fmaf(bf16_hi(xs[j]) + bf16_hi(zs[j]), bf16_hi(ys[j]), sum);
      } else {
        sum = fmaf(__builtin_bit_cast(float, xs[j]), __builtin_bit_cast(float, ys[j]), sum);
      }
    }
  }
#pragma unroll
  for (int o2 = 8; o2 > 0; o2 >>= 1) sum += __shfl_xor(sum, o2);
  if ((threadIdx.x & 15) == 0) {
    const float ls = p.lse_in[((long long)b * p.Hq + h) * p.Tq + t];
    reinterpret_cast<f32x2*>(p.stats)[row] = (f32x2){ls == -INFINITY ? ls : -ls * kLog2e, -sum};
  }
}

}  // namespace

hipError_t attn_combine_launch(const AttnParams& p, bool bf16, hipStream_t s) {
  return bf16 ? combine<uint16_t>(p, s) : combine<float>(p, s);
}

hipError_t attn_stats_launch(const AttnParams& p, bool bf16, hipStream_t s) {
  const long long n = ((long long)p.B * p.Hq * p.Tq + 15) / 16;
  if (bf16)
    hipLaunchKernelGGL((attn_stats_kernel<uint16_t>), grid_of(n), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((attn_stats_kernel<float>), grid_of(n), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace lstm
