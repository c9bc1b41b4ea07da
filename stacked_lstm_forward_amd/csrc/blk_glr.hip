// Gated linear recurrence, and its gradients (formulas: block/lstm_block.h).
//
// The steps of a channel are joined by a scan (affine maps c -> G + A c compose).  A
// workgroup has a chunk of the steps of CW * V channels of one sentence, rows of 128
// bytes: its lanes are CW groups of V neighbouring channels by 64 / CW slots in a wave,
// its waves more slots, and a slot is NS consecutive steps, which stay in registers.
//   1. every lane forms its slot's map from its steps;
//   2. maps are joined over the slots of a wave (shuffles) and over the waves (LDS),
//      and with the state that the chunk before ends with, which gives every slot the
//      state before it;
//   3. every lane goes through its steps again, from that state.
// So each value is read once, in one launch.  The gradients do the same twice: the
// states forwards, from the one that the forward kept for the chunk, the carry
// backwards.
// Bound by memory, beside a vector pipe at 70 % (forwards) and 54 %: 4 x 16384 x 1536
// (bf16, output gate) 469 us forwards and backwards, 4.8 TB/s (passes after each other; a
// kernel trace, which parts them, has 170 and 318, and 5 each to clear the chain's words);
// single steps by the launch (16 x 4096: 5.1 us), short sequences by loads, scan and
// stores after each other (64 x 100 x 512, fp32: 11 and 15 us).
#include "blk_common.h"
#include "blk_gate.h"

namespace lstm {
namespace {

constexpr int kWaves = 8;  // of a workgroup, at most
constexpr int kSteps = 8;  // NS

template <bool BF>
using Elem = typename Dt<BF>::T;

// How the work is laid out.
struct Plan {
  int cw, waves;
  long long tiles;  // of channels, of a sentence
  int chunk;        // steps
  int parts;        // chunks of T
};

// Channels of a lane: 8 bytes' worth forwards, two backwards, which has more to hold of each, and one in fp32 where
// the sequence is long: with two, gates and tanh spill, 7 registers with an output gate, 38 with both (32 x 500 x 4096:
// 437 us for 393, with tanh 528 for 420), with one, short sequences have fewer slots in a wave (64 x 100 x 512 without
// an output gate: 18.6 us for 16.0; between 100 and 500 steps, and short ones with gate and tanh, neither was measured).
// One where there are fewer.
int fwd_vector(const GlrParams& p, bool bf16) { return bf16 && p.H >= 4 ? 4 : !bf16 && p.H >= 2 ? 2 : 1; }
int bwd_vector(const GlrParams& p, bool bf16) { return p.H >= 2 && (bf16 || p.T <= 256) ? 2 : 1; }
constexpr int width_of(int V, int size) { return V * size * 16 >= 128 ? 16 : V * size * 32 >= 128 ? 32 : 64; }

Plan plan_of(const GlrParams& p, int V, int size) {
  Plan s;
  // rows of half the width where those of 128 bytes would leave a fifth of the lanes without channels of
  // their own (96 x 1446 x 71 forwards and backwards: 77 us for 65)
  const int wide = width_of(V, size), half = wide / 2;
  const long long at_wide = (p.H + V * wide - 1) / (V * wide), at_half = (p.H + V * half - 1) / (V * half);
  const int cw = at_half * 5 <= at_wide * 8 ? half : wide;
  s.cw = cw;
  s.tiles = cw == half ? at_half : at_wide;
  s.waves = 1;
  while (s.waves < kWaves && (long long)s.waves * (64 / cw) * kSteps < p.T) s.waves *= 2;
  s.chunk = s.waves * (64 / cw) * kSteps;
  s.parts = (int)(((long long)p.T + s.chunk - 1) / s.chunk);
  return s;
}
Plan fwd_plan(const GlrParams& p, bool bf16) { return plan_of(p, fwd_vector(p, bf16), bf16 ? 2 : 4); }
Plan bwd_plan(const GlrParams& p, bool bf16) { return plan_of(p, bwd_vector(p, bf16), bf16 ? 2 : 4); }

// ---- chunks that wait for one another's states --------------------------------
//
// A chunk's workgroup loads its steps and forms its map, and only then needs the state that the
// chunk before it ends with.  Chunks form groups of kGroup in the order of the scan: every chunk
// but a group's last publishes its map (which it knows without waiting), the last the state after
// it.  So a chunk takes the state that the group before ends with through the maps of its own
// group's chunks before it: always the same ones in the same order, whatever the timing, and only
// every kGroup-th wait follows on another (without groups 1 us a chunk: 243 us forwards and 564 us
// backwards at 1 x 65536 x 1536, bf16).  Both are 64 bits for each channel, written and read past the
// caches in one piece, so nothing else has to be ordered: A with its sign set beside G, or the sign
// beside the state; 0 is what has not been published.  The workgroups of a sentence's tile take its
// chunks by a ticket, earlier chunks first: whoever is waited for has started before, and itself
// waits for none that started later, so every wait ends.  (One that passes the caller's limit gives
// NaN and sets the error word.  A poll counts for a millisecond at most: a process whose turn on the
// device is over for longer has not waited.)
// A ticket for each tile, since one counter for all serves a workgroup every 11 ns.
constexpr int kGroup = 8;
static_assert(kGroup == kWaves, "a wave for each chunk of a group");
struct Chain {
  uint32_t* error;   // (in a line of its own)
  uint32_t* ticket;  // [B][tiles]
  uint64_t* word;    // [parts][B][tiles][CH]
  int parts;         // 1: nothing to wait for, none of the above
  long long limit;   // of a wait, ticks of 10 ns
};
constexpr long long kPoll = 100000;  // a millisecond

__global__ __launch_bounds__(256) void glr_clear_kernel(ulonglong2* p, long long n) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) p[i] = make_ulonglong2(0, 0);
}

// The i-th chunk's word for the ones behind it, before and after it knows its own state.
__device__ __forceinline__ void chain_word(uint64_t* w, float a, float g) {
  __hip_atomic_store(w, ((uint64_t)(__float_as_uint(a) | 0x80000000u) << 32) | __float_as_uint(g), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void chain_map(uint64_t* w, int i, const Map& m) {
  if (i % kGroup != kGroup - 1) chain_word(w, m.A, m.G);
}
__device__ __forceinline__ void chain_state(uint64_t* w, int i, float c) {
  if (i % kGroup == kGroup - 1) chain_word(w, 0.f, c);
}
// The words that the i-th chunk needs, gathered in LDS: wave q fetches that of the q-th chunk before it
// (a chunk that waits has kWaves = kGroup waves).  `before` is the word of the chunk before, `back` from
// one to the one before it.
template <int CH>
__device__ __forceinline__ void chain_gather(const Chain& chain, const uint64_t* before, long long back, int i,
                                             Map (&lds)[kGroup][CH]) {
  static_assert(CH <= 64, "a lane for each channel");
  const int q = threadIdx.x >> 6, j = threadIdx.x & 63, words = i % kGroup + (i >= kGroup);
  if (j < CH && q < words) {
    const uint64_t* w = before + q * back + j;
    long long last = wall_clock64(), waited = 0;
    uint64_t v;
    while (!(v = __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))) {
      const long long now = wall_clock64(), since = now - last;
      last = now;
      waited += since < kPoll ? since : kPoll;
      if (waited > chain.limit) {
        __hip_atomic_store(chain.error, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        v = 0x7fc000007fc00000ull;
        break;
      }
      __builtin_amdgcn_s_sleep(1);
    }
    lds[q][j] = {__uint_as_float((uint32_t)(v >> 32) & 0x7fffffffu), __uint_as_float((uint32_t)v)};
  }
  __syncthreads();
}
// The state before the i-th chunk of channel j; `first` is the one before the first chunk.
template <int CH>
__device__ __forceinline__ float chain_state_before(const Map (&lds)[kGroup][CH], int i, int j, float first) {
  float c = i < kGroup ? first : lds[i % kGroup][j].G;
  for (int q = i % kGroup - 1; q >= 0; --q) c = map_apply(lds[q][j], c);
  return c;
}

// Where a workgroup and a lane are.
template <int V, int CW>
struct Place {
  int b, n, tile, ch;  // sentence, its steps, the workgroup's tile, this lane's first channel
  int col, slot, wave;

  __device__ __forceinline__ void put(const GlrParams& p, unsigned tiles, unsigned blk) {
    b = (int)(blk / tiles);
    tile = (int)(blk % tiles);
    n = steps_of(p.lengths, b, p.T);
    const int lane = threadIdx.x & 63;
    wave = threadIdx.x >> 6;
    col = lane % CW;
    slot = wave * (64 / CW) + lane / CW;
    ch = channel(p, tile, col);
  }
  // The last lanes' vectors are moved back to end with the last channel: what two lanes have in
  // common they compute and write alike.
  static __device__ __forceinline__ int channel(const GlrParams& p, int tile, int col) {
    const long long c = ((long long)tile * CW + col) * V;
    return c + V <= p.H ? (int)c : p.H - V;
  }
  // of column j of the tile's CW * V
  __device__ __forceinline__ long long state(const GlrParams& p, int j) const {
    return (long long)b * p.H + channel(p, tile, j / V) + j % V;
  }
};

__device__ __forceinline__ Map shfl_up(const Map& m, int n) { return {__shfl_up(m.A, n), __shfl_up(m.G, n)}; }
__device__ __forceinline__ Map shfl_down(const Map& m, int n) { return {__shfl_down(m.A, n), __shfl_down(m.G, n)}; }

struct Yes {
  static constexpr bool value = true;
};
struct No {
  static constexpr bool value = false;
};

// A workgroup takes its place: the chunk, counted in the chain's order.
template <int V, int CW>
__device__ __forceinline__ int take(Place<V, CW>& at, const GlrParams& p, unsigned tiles, const Chain& chain, uint32_t* lds) {
  // Rows lie a multiple of the caches' channels apart: an XCD that had every 8th tile would use some of its
  // channels only (4 x 16384 x 1536: 180 us for 167).  So each has tiles beside one another, which also share
  // lines where a row is no multiple of 128 bytes (16 x 1000 x 700: 34 us for 24), and others after some rounds.
  const unsigned blocks = (unsigned)p.B * tiles, id = grid_block(), round = id / blocks;
  const unsigned turned = (id + round / kGroup) % blocks, xcd = turned % 8, more = blocks % 8;
  const unsigned at_block = xcd * (blocks / 8) + (xcd < more ? xcd : more) + turned / 8;
  at.put(p, tiles, at_block);
  if (round >= (unsigned)chain.parts) return chain.parts;  // a spare one
  if (chain.parts == 1) return 0;
  if (threadIdx.x == 0) *lds = atomicAdd(chain.ticket + at_block, 1u);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*lds);
}

// NS steps of a slot from t0.  FULL: all of them are the sentence's; else the last is read in
// the place of those behind it, and the values are not used.
template <bool FULL, bool BF, int V, int NS>
__device__ __forceinline__ void load_steps(Raw<BF, V> (&r)[NS], const Elem<BF>* p, int ch, long long stride, int t0, int n) {
  long long q = ch + (FULL || t0 < n ? t0 : n - 1) * stride;
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    r[j].load(p + q);
    if (FULL || t0 + j + 1 < n) q += stride;
  }
}

template <bool BF, int V, int CW, int NS, bool GATE>
__global__ __launch_bounds__(64 * kWaves, 4) void glr_fwd_kernel(GlrParams p, long long tiles, int keep, Chain chain) {
  typedef Elem<BF> E;
  constexpr int SLW = 64 / CW, CH = CW * V;
  __shared__ Map total[kWaves][CH];
  __shared__ Map words[kGroup][CH];
  __shared__ float before[kWaves][CH];
  Place<V, CW> at;
  __shared__ uint32_t ticket;
  const int part = take(at, p, tiles, chain, &ticket);
  if (part >= chain.parts) return;
  const int waves = blockDim.x >> 6, chunk = waves * SLW * NS, b = at.b, n = at.n;
  const E* f = (const E*)p.f + b * p.sf.b;
  const E* u = (const E*)p.u + b * p.su.b;
  const E* o = GATE ? (const E*)p.o + b * p.so.b : nullptr;
  E* y = (E*)p.y + b * p.sy.b;
  const int start = part * chunk, t0 = start + at.slot * NS;
  const int end = p.T - start < chunk ? p.T : start + chunk;
  if (start >= n) {  // behind the sentence's own
    Raw<BF, V> zero;
    zero.clear();
    for (int t = start + at.slot; t < end; t += waves * SLW) zero.store(y + at.ch + (long long)t * p.sy.t);
    if (n == 0 && part == 0 && p.cT)
      for (int j = threadIdx.x; j < CH; j += blockDim.x) p.cT[at.state(p, j)] = p.c0 ? p.c0[at.state(p, j)] : 0.f;
    return;
  }
  uint64_t* word = chain.word + (((long long)part * p.B + b) * tiles + at.tile) * CH;
  const long long word_step = (long long)p.B * tiles * CH;
  auto step = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    Raw<BF, V> rf[NS], ru[NS], ro[GATE ? NS : 1];
    load_steps<FULL>(rf, f, at.ch, p.sf.t, t0, n);
    load_steps<FULL>(ru, u, at.ch, p.su.t, t0, n);
    if constexpr (GATE) load_steps<FULL>(ro, o, at.ch, p.so.t, t0, n);
    float a[NS][V], add[NS][V];
    Map m[V];
#pragma unroll
    for (int i = 0; i < V; ++i) m[i] = {1.f, 0.f};
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const Gate g = gate_of<BF>(rf[j].get(i));
        const float v = ru[j].get(i);
        a[j][i] = g.open;
        add[j][i] = g.shut * (p.tanh ? tanh_of<BF>(v) : v);
        if (!FULL && t0 + j >= n) a[j][i] = 1.f, add[j][i] = 0.f;  // what is before stays
        m[i] = {m[i].A * a[j][i], __builtin_fmaf(a[j][i], m[i].G, add[j][i])};
      }
    // slots of the wave: maps of all up to each, then of those before it
    if constexpr (SLW > 1) {
#pragma unroll
      for (int d = 1; d < SLW; d *= 2)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const Map e = shfl_up(m[i], d * CW);
          if (at.slot % SLW >= d) m[i] = map_join(m[i], e);
        }
    }
    if (at.slot % SLW == SLW - 1)
#pragma unroll
      for (int i = 0; i < V; ++i) total[at.wave][at.col * V + i] = m[i];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (SLW > 1) m[i] = shfl_up(m[i], CW);
      if (at.slot % SLW == 0) m[i] = {1.f, 0.f};
    }
    __syncthreads();
    const bool more = start + chunk < n;
    if (chain.parts > 1) {
      if (more && threadIdx.x < CH) {
        Map m = total[0][threadIdx.x];
        for (int w = 1; w < waves; ++w) m = map_join(total[w][threadIdx.x], m);
        chain_map(word + threadIdx.x, part, m);
      }
      chain_gather(chain, word - word_step, -word_step, part, words);
    }
    for (int j = threadIdx.x; j < CH; j += blockDim.x) {
      float c = p.c0 ? p.c0[at.state(p, j)] : 0.f;
      if (part > 0) c = chain_state_before(words, part, j, c);
      for (int w = 0; w < waves; ++w) {
        before[w][j] = c;
        c = map_apply(total[w][j], c);
      }
      if (more)
        chain_state(word + j, part, c);
      else if (p.cT)
        p.cT[at.state(p, j)] = c;
    }
    __syncthreads();
    float c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = map_apply(m[i], before[at.wave][at.col * V + i]);
    if (p.reserve && t0 % keep == 0 && (FULL || t0 < n)) {
      float* r = p.reserve + ((long long)(t0 / keep) * p.B + b) * p.H + at.ch;
      __builtin_memcpy(r, c, V * 4);
    }
    long long q = at.ch + (long long)t0 * p.sy.t;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      float out[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        c[i] = __builtin_fmaf(a[j][i], c[i], add[j][i]);
        out[i] = c[i];
        if constexpr (GATE) out[i] *= sigmoid_of<BF>(ro[j].get(i));
        if (!FULL && t0 + j >= n) out[i] = 0.f;
      }
      if (FULL || t0 + j < p.T) {
        Raw<BF, V> r;
        r.set(out);
        r.store(y + q);
      }
      q += p.sy.t;
    }
  };
  if (start + chunk <= n)
    step(Yes());
  else
    step(No());
}

// One step of every sentence: nothing to join.
template <bool BF, int V, bool GATE>
__global__ __launch_bounds__(64) void glr_step_kernel(GlrParams p, long long tiles) {
  typedef Elem<BF> E;
  Place<V, 64> at;
  if (grid_block() >= p.B * tiles) return;
  at.put(p, tiles, grid_block());
  const int b = at.b;
  const long long bi = (long long)b * p.H + at.ch;
  float c[V], out[V];
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = 0.f, out[i] = 0.f;
  Raw<BF, V> f, u, o;
  f.load((const E*)p.f + b * p.sf.b + at.ch);
  u.load((const E*)p.u + b * p.su.b + at.ch);
  if constexpr (GATE) o.load((const E*)p.o + b * p.so.b + at.ch);
  if (p.c0) __builtin_memcpy(c, p.c0 + bi, V * 4);
  if (p.reserve) __builtin_memcpy(p.reserve + bi, c, V * 4);
  if (at.n > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const Gate g = gate_of<BF>(f.get(i));
      const float v = u.get(i);
      c[i] = __builtin_fmaf(g.open, c[i], g.shut * (p.tanh ? tanh_of<BF>(v) : v));
      out[i] = c[i];
      if constexpr (GATE) out[i] *= sigmoid_of<BF>(o.get(i));
    }
  }
  Raw<BF, V> r;
  r.set(out);
  r.store((E*)p.y + b * p.sy.b + at.ch);
  if (p.cT) __builtin_memcpy(p.cT + bi, c, V * 4);
}

template <bool BF, bool GBF, int V, int CW, int NS, bool GATE, bool TANH>
__global__ __launch_bounds__(64 * kWaves, 4) void glr_bwd_kernel(GlrParams p, long long tiles, Chain chain) {
  typedef Elem<BF> E;
  typedef Elem<GBF> G;
  constexpr int SLW = 64 / CW, CH = CW * V;
  __shared__ Map total[kWaves][CH];
  __shared__ Map words[kGroup][CH];
  __shared__ float total_g[kWaves][CH], before[kWaves][CH], after[kWaves][CH];
  Place<V, CW> at;
  __shared__ uint32_t ticket;
  const int part = chain.parts - 1 - take(at, p, tiles, chain, &ticket);
  if (part < 0) return;
  const int waves = blockDim.x >> 6, chunk = waves * SLW * NS, b = at.b, n = at.n;
  const E* f = (const E*)p.f + b * p.sf.b;
  const E* u = (const E*)p.u + b * p.su.b;
  const E* o = GATE ? (const E*)p.o + b * p.so.b : nullptr;
  const G* dy = (const G*)p.dy + b * p.sdy.b;
  G* df = (G*)p.df + b * p.sdf.b;
  G* du = (G*)p.du + b * p.sdu.b;
  G* dout = GATE ? (G*)p.dout_o + b * p.sdo.b : nullptr;
  const int start = part * chunk, t0 = start + at.slot * NS;
  const int end = p.T - start < chunk ? p.T : start + chunk;
  if (start >= n) {  // behind the sentence's own
    Raw<GBF, V> zero;
    zero.clear();
    for (long long t = start + at.slot; t < end; t += waves * SLW) {
      zero.store(df + at.ch + t * p.sdf.t);
      zero.store(du + at.ch + t * p.sdu.t);
      if constexpr (GATE) zero.store(dout + at.ch + t * p.sdo.t);
    }
    if (n == 0 && part == 0 && p.dc0)
      for (int j = threadIdx.x; j < CH; j += blockDim.x) p.dc0[at.state(p, j)] = p.dcT ? p.dcT[at.state(p, j)] : 0.f;
    return;
  }
  uint64_t* word = chain.word + (((long long)part * p.B + b) * tiles + at.tile) * CH;
  const long long word_step = (long long)p.B * tiles * CH;
  auto step = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    Raw<BF, V> rf[NS], ru[NS], ro[GATE ? NS : 1];
    Raw<GBF, V> rd[NS];
    load_steps<FULL>(rf, f, at.ch, p.sf.t, t0, n);
    load_steps<FULL>(ru, u, at.ch, p.su.t, t0, n);
    if constexpr (GATE) load_steps<FULL>(ro, o, at.ch, p.so.t, t0, n);
    load_steps<FULL>(rd, dy, at.ch, p.sdy.t, t0, n);
    // of each step: a, 1 - a, and what reaches c from y.  The candidate without a tanh and o's gate are taken
    // from the loaded values again where they are needed: two of a register beside one, and a gate is cheaper
    // than a register held.
    float a[NS][V], s[NS][V], up[NS][V], was[NS][V], tz[TANH ? NS : 1][V];
    auto z = [&](int j, int i) {
      if constexpr (TANH) return tz[j][i];
      const float v = ru[j].get(i);
      return FULL || t0 + j < n ? v : 0.f;
    };
    Map m[V], r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) m[i] = {1.f, 0.f};
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool in = FULL || t0 + j < n;
        const Gate g = gate_of<BF>(rf[j].get(i));
        a[j][i] = in ? g.open : 1.f, s[j][i] = in ? g.shut : 0.f;
        if constexpr (TANH) {
          const float v = ru[j].get(i);
          tz[j][i] = tanh_of<BF>(v);
          if (!in) tz[j][i] = 0.f;
        }
        up[j][i] = rd[j].get(i);
        if constexpr (GATE) up[j][i] *= sigmoid_of<BF>(ro[j].get(i));
        if (!in) up[j][i] = 0.f;
        m[i] = {m[i].A * a[j][i], __builtin_fmaf(a[j][i], m[i].G, s[j][i] * z(j, i))};
        // (step by step: mixed, the steps' intermediate values do not fit in the registers)
        if (i == V - 1) __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = {m[i].A, 0.f};
#pragma unroll
    for (int j = NS - 1; j >= 0; --j)
#pragma unroll
      for (int i = 0; i < V; ++i) r[i].G = a[j][i] * (up[j][i] + r[i].G);
    if constexpr (SLW > 1) {
#pragma unroll
      for (int d = 1; d < SLW; d *= 2)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const Map e = shfl_up(m[i], d * CW), l = shfl_down(r[i], d * CW);
          if (at.slot % SLW >= d) m[i] = map_join(m[i], e);
          if (at.slot % SLW + d < SLW) r[i] = map_join(r[i], l);
        }
    }
    if (at.slot % SLW == SLW - 1)
#pragma unroll
      for (int i = 0; i < V; ++i) total[at.wave][at.col * V + i] = m[i];
    if (at.slot % SLW == 0)
#pragma unroll
      for (int i = 0; i < V; ++i) total_g[at.wave][at.col * V + i] = r[i].G;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (SLW > 1) m[i] = shfl_up(m[i], CW), r[i] = shfl_down(r[i], CW);
      if (at.slot % SLW == 0) m[i] = {1.f, 0.f};
      if (at.slot % SLW == SLW - 1) r[i] = {1.f, 0.f};
    }
    __syncthreads();
    const int i = (n - 1) / chunk - part;  // in the chain, which begins at the sentence's last chunk
    if (chain.parts > 1) {
      if (part > 0 && threadIdx.x < CH) {
        Map m = {total[waves - 1][threadIdx.x].A, total_g[waves - 1][threadIdx.x]};
        for (int w = waves - 2; w >= 0; --w) m = map_join({total[w][threadIdx.x].A, total_g[w][threadIdx.x]}, m);
        chain_map(word + threadIdx.x, i, m);
      }
      chain_gather(chain, word + word_step, word_step, i, words);
    }
    for (int j = threadIdx.x; j < CH; j += blockDim.x) {
      float c = p.reserve[(long long)part * p.B * p.H + at.state(p, j)];
      for (int w = 0; w < waves; ++w) {
        before[w][j] = c;
        c = map_apply(total[w][j], c);
      }
      float d = p.dcT ? p.dcT[at.state(p, j)] : 0.f;
      if (i > 0) d = chain_state_before(words, i, j, d);
      for (int w = waves - 1; w >= 0; --w) {
        after[w][j] = d;
        d = __builtin_fmaf(total[w][j].A, d, total_g[w][j]);
      }
      if (part > 0)
        chain_state(word + j, i, d);
      else if (p.dc0)
        p.dc0[at.state(p, j)] = d;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      if constexpr (GATE) ro[j].hide();
      if constexpr (TANH) ru[j].hide();
    }
    // (what is made of a candidate is made again, not held)
    auto hide = [&]() {
      if constexpr (TANH && BF)
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) asm volatile("" : "+v"(tz[j][i]));
    };
    hide();
    float c[V], d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = map_apply(m[i], before[at.wave][at.col * V + i]);
      d[i] = map_apply(r[i], after[at.wave][at.col * V + i]);
    }
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        was[j][i] = c[i];
        c[i] = __builtin_fmaf(a[j][i], c[i], s[j][i] * z(j, i));
      }
    hide();
    long long qf = at.ch + (t0 + NS - 1) * p.sdf.t, qu = at.ch + (t0 + NS - 1) * p.sdu.t, qo = at.ch + (t0 + NS - 1) * p.sdo.t;
#pragma unroll
    for (int j = NS - 1; j >= 0; --j) {
      float vf[V], vu[V], vo[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (GATE) vo[i] = up[j][i] * c[i] * gate_of<BF>(ro[j].get(i)).shut;
        if (GATE && !FULL && t0 + j >= n) vo[i] = 0.f;
        c[i] = was[j][i];
        d[i] += up[j][i];
        vu[i] = d[i] * s[j][i];
        d[i] *= a[j][i];
        vf[i] = d[i] * ((c[i] - z(j, i)) * s[j][i]);
        if constexpr (TANH) vu[i] *= FULL || t0 + j < n ? tanh_slope<BF>(ru[j].get(i)) : 0.f;
      }
      if (FULL || t0 + j < p.T) {
        Raw<GBF, V> out;
        const bool behind = !FULL && t0 + j >= n;  // 0, also where c or d is not finite
        out.set(vf);
        if (behind) out.clear();
        out.store(df + qf);
        out.set(vu);
        if (behind) out.clear();
        out.store(du + qu);
        if constexpr (GATE) {
          out.set(vo);
          out.store(dout + qo);
        }
      }
      qf -= p.sdf.t, qu -= p.sdu.t, qo -= p.sdo.t;
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (start + chunk <= n)
    step(Yes());
  else
    step(No());
}

// The chain's 64-bit words: of the error word and the tickets (in lines of their own), and of the chunks.
constexpr int kErrorWords = 32;
long long ticket_words(const GlrParams& p, const Plan& s) { return kErrorWords + (p.B * s.tiles + 63) / 64 * 32; }
long long chain_words(const GlrParams& p, const Plan& s, int V) {
  return s.parts > 1 ? ticket_words(p, s) + s.parts * p.B * s.tiles * s.cw * V : 0;
}

// The chain's error word, tickets and words, cleared.
Chain chain_of(const GlrParams& p, const Plan& s, int V, hipStream_t stream) {
  if (s.parts > 1) {
    const long long n = chain_words(p, s, V) / 2;  // (a tile has an even number of channels)
    glr_clear_kernel<<<(int)(n / 256 < 1024 ? n / 256 + 1 : 1024), 256, 0, stream>>>((ulonglong2*)p.ws, n);
  }
  uint64_t* w = (uint64_t*)p.ws;
  return Chain{(uint32_t*)w, (uint32_t*)(w + kErrorWords), w + ticket_words(p, s), s.parts, p.wait};
}

template <bool BF, int V, bool GATE>
void fwd(const GlrParams& p, hipStream_t stream) {
  if (p.T == 1) {
    const long long tiles = (p.H + 64 * V - 1) / (64 * V);
    glr_step_kernel<BF, V, GATE><<<grid_of(p.B * tiles), 64, 0, stream>>>(p, tiles);
    return;
  }
  constexpr int CW = width_of(V, BF ? 2 : 4);
  const Plan s = fwd_plan(p, BF);
  const Chain chain = chain_of(p, s, V, stream);
  const dim3 grid = grid_of(s.parts * p.B * s.tiles);
  const int keep = bwd_plan(p, BF).chunk;
  if (s.cw == CW)
    glr_fwd_kernel<BF, V, CW, kSteps, GATE><<<grid, s.waves * 64, 0, stream>>>(p, s.tiles, keep, chain);
  else
    glr_fwd_kernel<BF, V, CW / 2, kSteps, GATE><<<grid, s.waves * 64, 0, stream>>>(p, s.tiles, keep, chain);
}

template <bool BF, bool GBF, int V, bool GATE, bool TANH>
void bwd(const GlrParams& p, hipStream_t stream) {
  constexpr int CW = width_of(V, BF ? 2 : 4);
  const Plan s = bwd_plan(p, BF);
  const Chain chain = chain_of(p, s, V, stream);
  const dim3 grid = grid_of(s.parts * p.B * s.tiles);
  if (s.cw == CW)
    glr_bwd_kernel<BF, GBF, V, CW, kSteps, GATE, TANH><<<grid, s.waves * 64, 0, stream>>>(p, s.tiles, chain);
  else
    glr_bwd_kernel<BF, GBF, V, CW / 2, kSteps, GATE, TANH><<<grid, s.waves * 64, 0, stream>>>(p, s.tiles, chain);
}

}  // namespace

size_t glr_reserve(const GlrParams& p, bool bf16) { return (size_t)bwd_plan(p, bf16).parts * p.B * p.H; }

size_t glr_workspace(const GlrParams& p, bool bf16) {
  const long long f = chain_words(p, fwd_plan(p, bf16), fwd_vector(p, bf16));
  const long long b = chain_words(p, bwd_plan(p, bf16), bwd_vector(p, bf16));
  return 8 * (size_t)(f > b ? f : b) + 256;
}

bool glr_waits(const GlrParams& p, bool bf16, bool train) {
  return train ? bwd_plan(p, bf16).parts > 1 : fwd_plan(p, bf16).parts > 1;
}

hipError_t glr_fwd_launch(const GlrParams& p, bool bf16, hipStream_t stream) {
  const bool one = fwd_vector(p, bf16) == 1;
#define CALL(BF, V) (p.o ? fwd<BF, V, true>(p, stream) : fwd<BF, V, false>(p, stream))
  if (bf16)
    one ? CALL(true, 1) : CALL(true, 4);
  else
    one ? CALL(false, 1) : CALL(false, 2);
#undef CALL
  return hipGetLastError();
}

hipError_t glr_bwd_launch(const GlrParams& p, bool bf16, bool grad_bf16, hipStream_t stream) {
  const bool one = bwd_vector(p, bf16) == 1;
#define CALL(BF, GBF, V)                                                                                     \
  (p.o ? (p.tanh ? bwd<BF, GBF, V, true, true>(p, stream) : bwd<BF, GBF, V, true, false>(p, stream))          \
       : (p.tanh ? bwd<BF, GBF, V, false, true>(p, stream) : bwd<BF, GBF, V, false, false>(p, stream)))
  if (!bf16)
    one ? CALL(false, false, 1) : CALL(false, false, 2);
  else if (grad_bf16)
    one ? CALL(true, true, 1) : CALL(true, true, 2);
  else
    one ? CALL(true, false, 1) : CALL(true, false, 2);
#undef CALL
  return hipGetLastError();
}

}  // namespace lstm
