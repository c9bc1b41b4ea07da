// C-ABI entry points of the block operators (host side): argument checks,
// parameters, launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "blk_clip.h"
#include "blk_common.h"
#include "block/lstm_block.h"  // include/ is on the include path

using namespace lstm;

namespace {

// Counts are held in 32 bits, and the kernels' signed counters step past them by less than 65536 (the recurrence's by
// a chunk of 512 steps at the most).  The norm's rows, which step by up to 6 x 256 x 64, are counted without a sign.
constexpr long long kMaxCount = (1ll << 31) - 65536;
constexpr int kMaxNorm = 16384;
constexpr long long kMaxElements = 1ll << 42;
constexpr int kMaxTensors = 1 << 20;
constexpr long long kWait = 2000000, kLongest = 1ll << 50;  // microseconds

bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool ws_ok(const void* ws) { return ws && aligned(ws, 256); }

// An output that begins where an input or another output does overlaps it, whatever the strides.
bool shared(std::initializer_list<const void*> outputs, std::initializer_list<const void*> inputs) {
  for (auto o = outputs.begin(); o != outputs.end(); ++o) {
    if (!*o) continue;
    for (const void* q : inputs)
      if (q == *o) return true;
    for (auto q = outputs.begin(); q != o; ++q)
      if (*q == *o) return true;
  }
  return false;
}

// Steps of an output lie apart: in either order of sentences and steps the inner stride holds a step, the
// outer one all that is inside.
bool apart(const lstm_seq_stride_t& s, long long B, long long T, long long W) {
  if (B == 1) return T == 1 || s.t >= W;
  if (T == 1) return s.b >= W;
  return (s.t >= W && s.b >= W && (s.b - W) / s.t >= T - 1) || (s.b >= W && s.t >= W && (s.t - W) / s.b >= B - 1);
}

bool alike(const lstm_seq_stride_t& a, const lstm_seq_stride_t& b) { return a.b == b.b && a.t == b.t; }

int size_of(int dtype) { return dtype == LSTM_BF16 ? 2 : 4; }

// What every description has: types, and counts that leave room.
lstm_status_t check_common(int B, int T, int W, int dtype, int grad_dtype, bool train) {
  if (B < 1 || T < 1 || W < 1) return LSTM_ERR_INVALID_ARG;
  if (dtype != LSTM_F32 && dtype != LSTM_BF16) return LSTM_ERR_INVALID_ARG;
  if (train && grad_dtype != LSTM_F32 && grad_dtype != LSTM_BF16) return LSTM_ERR_INVALID_ARG;
  if (train && dtype == LSTM_F32 && grad_dtype == LSTM_BF16) return LSTM_ERR_UNSUPPORTED;
  if ((long long)B * T > kMaxCount || (long long)B * W > kMaxCount) return LSTM_ERR_UNSUPPORTED;
  return LSTM_OK;
}

lstm_status_t check_norm(const lstm_norm_desc_t* d, bool train) {
  if (!d) return LSTM_ERR_INVALID_ARG;
  const lstm_status_t st = check_common(d->B, d->T, d->N, d->dtype, d->grad_dtype, train);
  if (st != LSTM_OK) return st;
  if (!(d->eps > 0.f) || std::isinf(d->eps)) return LSTM_ERR_INVALID_ARG;
  if (!apart(train ? d->dx : d->y, d->B, d->T, d->N)) return LSTM_ERR_INVALID_ARG;
  return d->N > kMaxNorm ? LSTM_ERR_UNSUPPORTED : LSTM_OK;
}

lstm_status_t check_glr(const lstm_glr_desc_t* d, bool train) {
  if (!d) return LSTM_ERR_INVALID_ARG;
  const lstm_status_t st = check_common(d->B, d->T, d->H, d->dtype, d->grad_dtype, train);
  if (st != LSTM_OK) return st;
  if (d->cand != LSTM_GLR_LINEAR && d->cand != LSTM_GLR_TANH) return LSTM_ERR_INVALID_ARG;
  if (train ? !apart(d->df, d->B, d->T, d->H) || !apart(d->du, d->B, d->T, d->H) : !apart(d->y, d->B, d->T, d->H))
    return LSTM_ERR_INVALID_ARG;
  // (the workgroups' tickets have 32 bits)
  return (long long)d->B * d->T > kMaxElements / d->H ? LSTM_ERR_UNSUPPORTED : LSTM_OK;
}

SeqStride stride(const lstm_seq_stride_t& s) { return SeqStride{s.b, s.t}; }

NormParams norm_params(const lstm_norm_desc_t* d) {
  NormParams p = {};
  p.B = d->B, p.T = d->T, p.N = d->N, p.eps = d->eps;
  p.sx = stride(d->x), p.sr = stride(d->r), p.ss = stride(d->s), p.sy = stride(d->y);
  p.sdy = stride(d->dy), p.sds = stride(d->ds), p.sdx = stride(d->dx);
  return p;
}

GlrParams glr_params(const lstm_glr_desc_t* d) {
  GlrParams p = {};
  p.B = d->B, p.T = d->T, p.H = d->H, p.tanh = d->cand == LSTM_GLR_TANH;
  p.sf = stride(d->f), p.su = stride(d->u), p.so = stride(d->o), p.sy = stride(d->y);
  p.sdy = stride(d->dy), p.sdf = stride(d->df), p.sdu = stride(d->du), p.sdo = stride(d->dout_o);
  const long long us = d->wait_timeout_us ? d->wait_timeout_us : kWait;
  p.wait = us < 0 ? -1 : us < kLongest ? us * 100 : kLongest * 100;
  return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Chunks of all tensors; -1 if the list is invalid.
long long clip_chunks(const lstm_clip_tensor_t* t, int n) {
  if (!t || n < 1 || n > kMaxTensors) return -1;
  long long chunks = 0, total = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].dtype != LSTM_F32 && t[i].dtype != LSTM_BF16) return -1;
    if (t[i].count < 0 || t[i].count > kMaxElements - total) return -1;
    const int size = size_of(t[i].dtype);
    if ((t[i].count > 0 && !t[i].src) || !aligned(t[i].src, size) || !aligned(t[i].dst, size)) return -1;
    total += t[i].count;
    chunks += (t[i].count + kClipChunk - 1) / kClipChunk;
  }
  return chunks;
}

int clip_blocks(long long chunks) { return chunks < 1 ? 1 : chunks < kClipBlocks ? (int)chunks : kClipBlocks; }

// The table: entries, the workgroups' spans, their partial sums.
size_t clip_span_at(int n) { return round256((size_t)n * sizeof(ClipEntry)); }
size_t clip_part_at(int n, int blocks) { return clip_span_at(n) + round256(blocks * sizeof(int2)); }

ClipParams clip_params(int n, long long chunks, void* table) {
  ClipParams p = {};
  p.n = n, p.chunks = chunks, p.blocks = clip_blocks(chunks);
  p.table = (const ClipEntry*)table, p.span = (const int2*)((char*)table + clip_span_at(n));
  p.part = (double*)((char*)table + clip_part_at(n, p.blocks));
  return p;
}

}  // namespace

extern "C" {

lstm_status_t lstm_norm_validate(const lstm_norm_desc_t* d, int train) { return check_norm(d, train != 0); }

size_t lstm_norm_bwd_workspace_size(const lstm_norm_desc_t* d) {
  if (check_norm(d, true) != LSTM_OK) return 0;
  return round256(norm_bwd_parts(norm_params(d)) * sizeof(float));
}

lstm_status_t lstm_norm_fwd(const lstm_norm_desc_t* d, const void* x, const void* r, const void* w, const void* b,
                            const int32_t* lengths, void* s, void* y, float* mean, float* rstd, hipStream_t stream) {
  const lstm_status_t st = check_norm(d, false);
  if (st != LSTM_OK) return st;
  if (!x || !y || (s && (!r || !apart(d->s, d->B, d->T, d->N)))) return LSTM_ERR_INVALID_ARG;
  const int size = size_of(d->dtype);
  for (const void* q : {x, r, w, b, (const void*)s, (const void*)y})
    if (!aligned(q, size)) return LSTM_ERR_INVALID_ARG;
  if (!aligned(lengths, 4) || !aligned(mean, 4) || !aligned(rstd, 4)) return LSTM_ERR_INVALID_ARG;
  if (shared({y, mean, rstd}, {x, r, w, b, lengths, s}) || shared({s}, {w, b, lengths})) return LSTM_ERR_INVALID_ARG;
  // (a step is read before its sum is written, another's place is not)
  if (s && ((s == x && !alike(d->s, d->x)) || (s == r && !alike(d->s, d->r)))) return LSTM_ERR_INVALID_ARG;
  NormParams p = norm_params(d);
  p.x = x, p.r = r, p.w = w, p.b = b, p.lengths = lengths, p.s = s, p.y = y, p.mean = mean, p.rstd = rstd;
  return norm_fwd_launch(p, d->dtype == LSTM_BF16, stream) == hipSuccess ? LSTM_OK : LSTM_ERR_HIP;
}

lstm_status_t lstm_norm_bwd(const lstm_norm_desc_t* d, const void* s, const void* w, const int32_t* lengths,
                            const float* mean, const float* rstd, const void* dy, const void* ds, void* dx, float* dw,
                            float* db, void* ws, hipStream_t stream) {
  const lstm_status_t st = check_norm(d, true);
  if (st != LSTM_OK) return st;
  if (!s || !mean || !rstd || !dy || !dx) return LSTM_ERR_INVALID_ARG;
  const int size = size_of(d->dtype), gsize = size_of(d->grad_dtype);
  if (!aligned(s, size) || !aligned(w, size) || !aligned(dy, gsize) || !aligned(ds, gsize) || !aligned(dx, gsize))
    return LSTM_ERR_INVALID_ARG;
  for (const void* q : {(const void*)lengths, (const void*)mean, (const void*)rstd, (const void*)dw, (const void*)db})
    if (!aligned(q, 4)) return LSTM_ERR_INVALID_ARG;
  if (!ws_ok(ws)) return LSTM_ERR_WORKSPACE;
  if (shared({dx, dw, db, ws}, {s, w, lengths, mean, rstd, dy, ds})) return LSTM_ERR_INVALID_ARG;
  NormParams p = norm_params(d);
  p.x = s, p.w = w, p.lengths = lengths, p.mean = const_cast<float*>(mean), p.rstd = const_cast<float*>(rstd);
  p.dy = dy, p.ds = ds, p.dx = dx, p.dw = dw, p.db = db, p.part = (float*)ws;
  return norm_bwd_launch(p, d->dtype == LSTM_BF16, d->grad_dtype == LSTM_BF16, stream) == hipSuccess ? LSTM_OK
                                                                                                     : LSTM_ERR_HIP;
}

lstm_status_t lstm_glr_validate(const lstm_glr_desc_t* d, int train) { return check_glr(d, train != 0); }

size_t lstm_glr_reserve_size(const lstm_glr_desc_t* d) {
  if (check_glr(d, false) != LSTM_OK) return 0;
  return round256(glr_reserve(glr_params(d), d->dtype == LSTM_BF16) * sizeof(float));
}

size_t lstm_glr_workspace_size(const lstm_glr_desc_t* d) {
  if (check_glr(d, false) != LSTM_OK) return 0;
  return round256(glr_workspace(glr_params(d), d->dtype == LSTM_BF16));
}

lstm_status_t lstm_glr_fwd(const lstm_glr_desc_t* d, const void* f, const void* u, const void* o, const float* c0,
                           const int32_t* lengths, void* y, float* cT, void* reserve, void* ws, hipStream_t stream) {
  const lstm_status_t st = check_glr(d, false);
  if (st != LSTM_OK) return st;
  if (!f || !u || !y) return LSTM_ERR_INVALID_ARG;
  const int size = size_of(d->dtype);
  for (const void* q : {f, u, o, (const void*)y})
    if (!aligned(q, size)) return LSTM_ERR_INVALID_ARG;
  if (!aligned(lengths, 4) || !aligned(c0, 4) || !aligned(cT, 4)) return LSTM_ERR_INVALID_ARG;
  if (!aligned(reserve, 256) || !ws_ok(ws)) return LSTM_ERR_WORKSPACE;
  if (shared({y, cT, reserve, ws}, {f, u, o, c0, lengths})) return LSTM_ERR_INVALID_ARG;
  GlrParams p = glr_params(d);
  p.f = f, p.u = u, p.o = o, p.c0 = c0, p.lengths = lengths, p.y = y, p.cT = cT, p.reserve = (float*)reserve;
  p.ws = ws;
  return glr_fwd_launch(p, d->dtype == LSTM_BF16, stream) == hipSuccess ? LSTM_OK : LSTM_ERR_HIP;
}

lstm_status_t lstm_glr_bwd(const lstm_glr_desc_t* d, const void* f, const void* u, const void* o, const float* c0,
                           const int32_t* lengths, const void* reserve, const void* dy, const float* dcT, void* df,
                           void* du, void* dout_o, float* dc0, void* ws, hipStream_t stream) {
  const lstm_status_t st = check_glr(d, true);
  if (st != LSTM_OK) return st;
  if (!f || !u || !dy || !df || !du) return LSTM_ERR_INVALID_ARG;
  if (o && (!dout_o || !apart(d->dout_o, d->B, d->T, d->H))) return LSTM_ERR_INVALID_ARG;
  const int size = size_of(d->dtype), gsize = size_of(d->grad_dtype);
  if (!aligned(f, size) || !aligned(u, size) || !aligned(o, size)) return LSTM_ERR_INVALID_ARG;
  for (const void* q : {dy, (const void*)df, (const void*)du, (const void*)dout_o})
    if (!aligned(q, gsize)) return LSTM_ERR_INVALID_ARG;
  for (const void* q : {(const void*)lengths, (const void*)c0, (const void*)dcT, (const void*)dc0})
    if (!aligned(q, 4)) return LSTM_ERR_INVALID_ARG;
  if (!ws_ok(reserve) || !ws_ok(ws)) return LSTM_ERR_WORKSPACE;
  if (shared({df, du, o ? dout_o : nullptr, dc0, ws}, {f, u, o, c0, lengths, reserve, dy, dcT})) return LSTM_ERR_INVALID_ARG;
  GlrParams p = glr_params(d);
  p.f = f, p.u = u, p.o = o, p.c0 = c0, p.lengths = lengths, p.reserve = (float*)const_cast<void*>(reserve);
  p.dy = dy, p.dcT = dcT, p.df = df, p.du = du, p.dout_o = dout_o, p.dc0 = dc0, p.ws = ws;
  return glr_bwd_launch(p, d->dtype == LSTM_BF16, d->grad_dtype == LSTM_BF16, stream) == hipSuccess ? LSTM_OK
                                                                                                    : LSTM_ERR_HIP;
}

lstm_status_t lstm_glr_last_error(const lstm_glr_desc_t* d, int train, const void* ws, hipStream_t stream) {
  const lstm_status_t st = check_glr(d, train != 0);
  if (st != LSTM_OK) return st;
  if (!ws_ok(ws)) return LSTM_ERR_WORKSPACE;
  if (hipStreamSynchronize(stream) != hipSuccess) return LSTM_ERR_HIP;
  if (!glr_waits(glr_params(d), d->dtype == LSTM_BF16, train != 0)) return LSTM_OK;
  uint32_t v = 0;
  if (hipMemcpy(&v, ws, sizeof(v), hipMemcpyDeviceToHost) != hipSuccess) return LSTM_ERR_HIP;
  return v == 0 ? LSTM_OK : LSTM_ERR_BARRIER_TIMEOUT;
}

size_t lstm_clip_table_size(const lstm_clip_tensor_t* tensors, int32_t n) {
  const long long chunks = clip_chunks(tensors, n);
  return chunks < 0 ? 0 : clip_part_at(n, clip_blocks(chunks)) + round256(clip_blocks(chunks) * sizeof(double));
}

lstm_status_t lstm_clip_table(const lstm_clip_tensor_t* tensors, int32_t n, void* table, hipStream_t stream) {
  const long long chunks = clip_chunks(tensors, n);
  if (chunks < 0) return LSTM_ERR_INVALID_ARG;
  if (!ws_ok(table)) return LSTM_ERR_WORKSPACE;
  long long first = 0;
  ClipTableArgs a;
  a.table = (ClipEntry*)table;
  for (int i = 0; i < n; i += kClipEntries) {
    a.at = i, a.n = n - i < kClipEntries ? n - i : kClipEntries;
    for (int j = 0; j < a.n; ++j) {
      const lstm_clip_tensor_t& t = tensors[i + j];
      a.entry[j] = ClipEntry{t.src, t.dst, t.count, first, t.dtype == LSTM_BF16, 0};
      first += (t.count + kClipChunk - 1) / kClipChunk;
    }
    if (clip_table_launch(a, stream) != hipSuccess) return LSTM_ERR_HIP;
  }
  const ClipParams p = clip_params(n, chunks, table);
  return clip_span_launch(p, const_cast<int2*>(p.span), stream) == hipSuccess ? LSTM_OK : LSTM_ERR_HIP;
}

lstm_status_t lstm_clip(const lstm_clip_tensor_t* tensors, int32_t n, void* table, double max_norm, double eps,
                        float* out, hipStream_t stream) {
  const long long chunks = clip_chunks(tensors, n);
  if (chunks < 0) return LSTM_ERR_INVALID_ARG;
  if (!(max_norm >= 0) || !(eps >= 0) || std::isinf(eps) || !out || !aligned(out, 4)) return LSTM_ERR_INVALID_ARG;
  if (!ws_ok(table)) return LSTM_ERR_WORKSPACE;
  ClipParams p = clip_params(n, chunks, table);
  p.out = out, p.max_norm = max_norm, p.eps = eps;
  return clip_launch(p, stream) == hipSuccess ? LSTM_OK : LSTM_ERR_HIP;
}

}  // extern "C"
