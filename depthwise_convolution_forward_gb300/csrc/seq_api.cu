// C ABI of the sequence operators (gconv_seq.h): argument validation and
// launch.  Everything here runs on the host; the arithmetic runs in scan.cu,
// conv1d.cu, normq.cu and mmq.cu.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>

#include "seq.h"

namespace gconv {
namespace {

constexpr int64_t kMaxExtent = (int64_t)1 << 40;
constexpr int64_t kMaxColumns = (int64_t)1 << 36;  // channels of all sequences (keeps launch grids in range)

gconv_status check_dtype(gconv_dtype dt) {
  if (dt != GCONV_F32 && dt != GCONV_F16 && dt != GCONV_BF16)
    return set_last_error(GCONV_ERR_UNSUPPORTED, "unknown dtype %d", (int)dt);
  return GCONV_OK;
}

// A buffer as a call sees it: `row` = 0 for a packed one of `bytes` bytes,
// else a strided [B, T, D] tensor whose two strides are known, so that ranges of
// the columns, tokens or sequences of one larger tensor can be told apart from
// buffers that overlap.
struct Span {
  const void* p;
  int64_t bytes;       // from the first to past the last byte
  int64_t row, width;  // packed: 0; else bytes between tokens, bytes of one token
  int64_t batch;       // bytes between sequences
  int64_t run;         // bytes from the first to past the last row along the smaller stride
};

Span packed(const void* p, int64_t bytes) { return {p, p ? bytes : 0, 0, 0, 0, 0}; }

Span strided(const void* p, int64_t B, int64_t T, int64_t D, SeqStride s, int es) {
  const int64_t run = s.t <= s.b ? (T - 1) * s.t + D : (B - 1) * s.b + D;
  return {p, p ? ((B - 1) * s.b + (T - 1) * s.t + D) * es : 0, s.t * es, D * es, s.b * es, run * es};
}

// Whether pieces of la bytes at every multiple of `pitch` from a and pieces of lb
// bytes at every multiple of it from b lie beside each other.
bool beside(uintptr_t a, int64_t la, uintptr_t b, int64_t lb, int64_t pitch) {
  const int64_t d = b >= a ? (int64_t)((b - a) % (uintptr_t)pitch) : (pitch - (int64_t)((a - b) % (uintptr_t)pitch)) % pitch;
  return d >= la && d <= pitch - lb;
}

bool touch(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  if (a0 >= b0 + (uintptr_t)b.bytes || b0 >= a0 + (uintptr_t)a.bytes) return false;
  // Interleaved ranges of one larger tensor, which have the same strides.  Tokens or
  // sequences: a run of rows along the smaller stride is a piece, the larger stride
  // the pitch.  Columns: a row is a piece, the smaller stride the pitch, of which the
  // larger one is a multiple.
  if (a.row > 0 && a.batch > 0 && a.row == b.row && a.batch == b.batch) {
    const int64_t lo = a.row < a.batch ? a.row : a.batch, hi = a.row < a.batch ? a.batch : a.row;
    if (beside(a0, a.run, b0, b.run, hi) || (hi % lo == 0 && beside(a0, a.width, b0, b.width, lo))) return false;
  }
  return true;
}

// Whether any output overlaps an input or another output.
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (touch(*o, i)) return true;
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (touch(*o, *q)) return true;
  }
  return false;
}

gconv_status check_extents(int64_t B, int64_t T, int32_t D) {
  if (B < 1 || T < 1) return set_last_error(GCONV_ERR_INVALID_ARG, "B and T must be >= 1");
  if (D < 1 || D > GCONV_SEQ_MAX_D)  // whole blocks of up to 128 channels stay within 31 bits
    return set_last_error(GCONV_ERR_INVALID_ARG, "D must be 1 ... %d", GCONV_SEQ_MAX_D);
  if (B > kMaxExtent || T > kMaxExtent || (double)B * D > (double)kMaxColumns || (double)B * (double)T * (double)D > 1e18)
    return set_last_error(GCONV_ERR_INVALID_ARG, "tensor too large");
  return GCONV_OK;
}

// Strides of a [B, T, D] tensor: {0, 0} is packed; rows must not overlap.
gconv_status check_stride(const int64_t in[2], int64_t B, int64_t T, int64_t D, const char* what, SeqStride* out) {
  SeqStride s{in[0], in[1]};
  if (s.b == 0 && s.t == 0) s = {T * D, D};
  if (s.b < 0 || s.t < 0 || (double)(B - 1) * (double)s.b + (double)(T - 1) * (double)s.t + (double)D > 1e18)
    return set_last_error(GCONV_ERR_INVALID_ARG, "strides of %s out of range", what);
  // A stride that no element uses may be anything; it takes the other's value.
  if (B == 1 && T == 1) s = {D, D};
  else if (B == 1) s.b = s.t;
  else if (T == 1) s.t = s.b;
  const bool batch_major = (T == 1 || s.t >= D) && (B == 1 || (double)s.b >= (double)(T - 1) * s.t + D);
  const bool time_major = (B == 1 || s.b >= D) && (T == 1 || (double)s.t >= (double)(B - 1) * s.b + D);
  if (!batch_major && !time_major)
    return set_last_error(GCONV_ERR_INVALID_ARG, "rows of %s overlap one another", what);
  *out = s;
  return GCONV_OK;
}

gconv_status prepare(struct CUstream_st* stream, gconv_dtype dt, LaunchArgs* a, DeviceInfo* dev) {
  int* status = nullptr;
  const cudaError_t e = current_device(dev, &status);
  if (e != cudaSuccess) return set_last_error(GCONV_ERR_CUDA, "device query failed: %s", cudaGetErrorString(e));
  *a = LaunchArgs{};
  a->dt = (DType)dt;
  a->stream = reinterpret_cast<cudaStream_t>(stream);
  a->status = status;
  a->wait_limit_ns = 2000000000ull;
  a->pdl = true;
  return GCONV_OK;
}

gconv_status done(cudaError_t e) {
  if (e != cudaSuccess) return set_last_error(GCONV_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
  return GCONV_OK;
}

gconv_status check_workspace(const void* ws, int64_t have, int64_t need) {
  if (ws == nullptr || have < need || (reinterpret_cast<uintptr_t>(ws) & 15))
    return set_last_error(GCONV_ERR_INVALID_ARG, "workspace must be 16-byte aligned and hold %lld bytes",
                          (long long)need);
  return GCONV_OK;
}

gconv_status check_conv1d(const gconv_conv1d_problem* p, gconv_dtype dt, ConvSeqArgs* c) {
  if (p == nullptr) return set_last_error(GCONV_ERR_INVALID_ARG, "problem pointer is NULL");
  if (p->reserved != 0) return set_last_error(GCONV_ERR_INVALID_ARG, "reserved field must be 0");
  gconv_status s = check_extents(p->B, p->T, p->D);
  if (s != GCONV_OK) return s;
  if (p->K < 1 || p->K > GCONV_CONV1D_MAX_K)
    return set_last_error(GCONV_ERR_INVALID_ARG, "K must be 1 ... %d", GCONV_CONV1D_MAX_K);
  if (p->act != 0 && p->act != 1) return set_last_error(GCONV_ERR_INVALID_ARG, "act must be 0 or 1");
  s = check_dtype(dt);
  if (s != GCONV_OK) return s;
  *c = ConvSeqArgs{};
  c->B = p->B, c->T = p->T, c->D = p->D, c->K = p->K, c->act = p->act;
  s = check_stride(p->x_stride, p->B, p->T, p->D, "x", &c->sx);
  if (s != GCONV_OK) return s;
  return check_stride(p->y_stride, p->B, p->T, p->D, "y", &c->sy);
}

gconv_status check_scan(const gconv_scan_problem* p, gconv_dtype dt, ScanArgs* a) {
  if (p == nullptr) return set_last_error(GCONV_ERR_INVALID_ARG, "problem pointer is NULL");
  gconv_status s = check_extents(p->B, p->T, p->D);
  if (s != GCONV_OK) return s;
  if (!(p->decay > 0.f) || !std::isfinite(p->decay))
    return set_last_error(GCONV_ERR_INVALID_ARG, "decay must be positive and finite");
  s = check_dtype(dt);
  if (s != GCONV_OK) return s;
  *a = ScanArgs{};
  a->B = p->B, a->T = p->T, a->D = p->D, a->decay = p->decay;
  const int64_t* in[4] = {p->x_stride, p->r_stride, p->i_stride, p->y_stride};
  const char* what[4] = {"x", "r", "i", "y"};
  SeqStride* out[4] = {&a->sx, &a->sr, &a->si, &a->sy};
  for (int k = 0; k < 4; ++k) {
    s = check_stride(in[k], p->B, p->T, p->D, what[k], out[k]);
    if (s != GCONV_OK) return s;
  }
  return GCONV_OK;
}

gconv_status check_norm(const gconv_norm_problem* p, gconv_dtype dt, NormArgs* n) {
  if (p == nullptr) return set_last_error(GCONV_ERR_INVALID_ARG, "problem pointer is NULL");
  if (p->reserved != 0) return set_last_error(GCONV_ERR_INVALID_ARG, "reserved field must be 0");
  if (p->rows < 0 || p->rows > 0x7fffffff)
    return set_last_error(GCONV_ERR_INVALID_ARG, "rows must be 0 ... 2^31 - 1");
  if (p->D < 1 || p->D > GCONV_NORM_MAX_D)
    return set_last_error(GCONV_ERR_INVALID_ARG, "D must be 1 ... %d", GCONV_NORM_MAX_D);
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps))
    return set_last_error(GCONV_ERR_INVALID_ARG, "eps must be finite and not negative");
  const int64_t* in[3] = {&p->x_stride, &p->residual_stride, &p->y_stride};
  *n = NormArgs{};
  int64_t* out[3] = {&n->sx, &n->sr, &n->sy};
  for (int k = 0; k < 3; ++k) {
    if (*in[k] != 0 && (*in[k] < p->D || (double)p->rows * (double)*in[k] > 1e18))
      return set_last_error(GCONV_ERR_INVALID_ARG, "a row stride is below D or out of range");
    *out[k] = *in[k] ? *in[k] : p->D;
  }
  n->rows = p->rows, n->D = p->D, n->eps = p->eps;
  return check_dtype(dt);
}

}  // namespace
}  // namespace gconv

using namespace gconv;

extern "C" {

gconv_status gconv_causal_conv1d_fwd(const void* x, const void* w, const void* bias, const void* state_in,
                                     const int32_t* lens, void* y, void* state_out, const gconv_conv1d_problem* p,
                                     gconv_dtype dt, struct CUstream_st* stream) {
  ConvSeqArgs c;
  gconv_status s = check_conv1d(p, dt, &c);
  if (s != GCONV_OK) return s;
  if (x == nullptr || w == nullptr || y == nullptr)
    return set_last_error(GCONV_ERR_INVALID_ARG, "x, w and y must not be NULL");
  if (c.K == 1) state_in = nullptr, state_out = nullptr;
  const int es = dtype_bytes((DType)dt);
  const int64_t sb = c.B * (c.K - 1) * c.D * es;
  const Span xs = strided(x, c.B, c.T, c.D, c.sx, es), ys = strided(y, c.B, c.T, c.D, c.sy, es);
  const Span ws = packed(w, (int64_t)c.D * c.K * es), bs = packed(bias, (int64_t)c.D * es), ls = packed(lens, c.B * 4);
  if (clash({ys, packed(state_out, sb)}, {xs, ws, bs, ls, packed(state_in == state_out ? nullptr : state_in, sb)}) ||
      touch(ys, packed(state_in, sb)))
    return set_last_error(GCONV_ERR_INVALID_ARG, "an output overlaps an input or another output");
  LaunchArgs a;
  DeviceInfo dev;
  s = prepare(stream, dt, &a, &dev);
  if (s != GCONV_OK) return s;
  c.x = x, c.w = w, c.bias = bias, c.state_in = state_in, c.lens = lens, c.y = y, c.state_out = state_out;
  return done(conv1d_fwd_launch(c, a, dev));
}

gconv_status gconv_causal_conv1d_bwd_workspace_size(const gconv_conv1d_problem* p, gconv_dtype dt, int64_t* bytes) {
  ConvSeqArgs c;
  gconv_status s = check_conv1d(p, dt, &c);
  if (s != GCONV_OK) return s;
  if (bytes == nullptr) return set_last_error(GCONV_ERR_INVALID_ARG, "bytes pointer is NULL");
  *bytes = conv1d_bwd_workspace_bytes(c.B, c.T, c.D, c.K);
  return GCONV_OK;
}

gconv_status gconv_causal_conv1d_bwd(const void* dy, const void* dstate_out, const void* x, const void* w,
                                     const void* bias, const void* state_in, const int32_t* lens, void* dx, void* dw,
                                     void* dbias, void* dstate_in, const gconv_conv1d_problem* p, gconv_dtype dt,
                                     void* workspace, int64_t workspace_bytes, struct CUstream_st* stream) {
  ConvSeqArgs c;
  gconv_status s = check_conv1d(p, dt, &c);
  if (s != GCONV_OK) return s;
  if (dy == nullptr || x == nullptr || w == nullptr || dx == nullptr || dw == nullptr)
    return set_last_error(GCONV_ERR_INVALID_ARG, "dy, x, w, dx and dw must not be NULL");
  const int64_t need = conv1d_bwd_workspace_bytes(c.B, c.T, c.D, c.K);
  s = check_workspace(workspace, workspace_bytes, need);
  if (s != GCONV_OK) return s;
  if (c.K == 1) state_in = nullptr, dstate_out = nullptr, dstate_in = nullptr;
  const int es = dtype_bytes((DType)dt);
  const int64_t sb = c.B * (c.K - 1) * c.D * es, wb = (int64_t)c.D * c.K * es, bb = (int64_t)c.D * es;
  if (clash({strided(dx, c.B, c.T, c.D, c.sx, es), packed(dw, wb), packed(dbias, bb), packed(dstate_in, sb),
             packed(workspace, need)},
            {strided(dy, c.B, c.T, c.D, c.sy, es), strided(x, c.B, c.T, c.D, c.sx, es), packed(w, wb),
             packed(bias, bb), packed(state_in, sb), packed(dstate_out, sb), packed(lens, c.B * 4)}))
    return set_last_error(GCONV_ERR_INVALID_ARG, "an output or the workspace overlaps another buffer");
  LaunchArgs a;
  DeviceInfo dev;
  s = prepare(stream, dt, &a, &dev);
  if (s != GCONV_OK) return s;
  c.dy = dy, c.dstate_out = dstate_out, c.x = x, c.w = w, c.bias = bias, c.state_in = state_in, c.lens = lens;
  c.dx = dx, c.dw = dw, c.dbias = dbias, c.dstate_in = dstate_in, c.ws = static_cast<float*>(workspace);
  return done(conv1d_bwd_launch(c, a, dev));
}

gconv_status gconv_gated_scan_fwd(const void* x, const void* r, const void* i, const float* lam, const float* h0,
                                  const int32_t* lens, void* y, float* hT, void* saved, const gconv_scan_problem* p,
                                  gconv_dtype dt, struct CUstream_st* stream) {
  ScanArgs q;
  gconv_status s = check_scan(p, dt, &q);
  if (s != GCONV_OK) return s;
  if (x == nullptr || r == nullptr || i == nullptr || lam == nullptr || y == nullptr)
    return set_last_error(GCONV_ERR_INVALID_ARG, "x, r, i, lam and y must not be NULL");
  if (reinterpret_cast<uintptr_t>(saved) & 15)
    return set_last_error(GCONV_ERR_INVALID_ARG, "saved must be 16-byte aligned");
  const int es = dtype_bytes((DType)dt);
  const int64_t hb = q.B * (int64_t)q.D * 4;
  const Span h0s = packed(h0, hb), ys = strided(y, q.B, q.T, q.D, q.sy, es);
  const Span svs = packed(saved, scan_saved_bytes(q.B, q.T, q.D));
  if (clash({ys, packed(hT, hb), svs},
            {strided(x, q.B, q.T, q.D, q.sx, es), strided(r, q.B, q.T, q.D, q.sr, es),
             strided(i, q.B, q.T, q.D, q.si, es), packed(lam, (int64_t)q.D * 4), packed(lens, q.B * 4),
             hT == h0 ? packed(nullptr, 0) : h0s}) ||
      touch(ys, h0s) || touch(svs, h0s))
    return set_last_error(GCONV_ERR_INVALID_ARG, "an output overlaps an input or another output");
  LaunchArgs a;
  DeviceInfo dev;
  s = prepare(stream, dt, &a, &dev);
  if (s != GCONV_OK) return s;
  q.x = x, q.r = r, q.i = i, q.lam = lam, q.h0 = h0, q.lens = lens, q.y = y, q.hT = hT;
  q.saved = static_cast<float*>(saved);
  return done(scan_fwd_launch(q, a, dev));
}

gconv_status gconv_gated_scan_saved_size(const gconv_scan_problem* p, gconv_dtype dt, int64_t* bytes) {
  ScanArgs q;
  gconv_status s = check_scan(p, dt, &q);
  if (s != GCONV_OK) return s;
  if (bytes == nullptr) return set_last_error(GCONV_ERR_INVALID_ARG, "bytes pointer is NULL");
  *bytes = scan_saved_bytes(q.B, q.T, q.D);
  return GCONV_OK;
}

gconv_status gconv_gated_scan_bwd_workspace_size(const gconv_scan_problem* p, gconv_dtype dt, int64_t* bytes) {
  ScanArgs q;
  gconv_status s = check_scan(p, dt, &q);
  if (s != GCONV_OK) return s;
  if (bytes == nullptr) return set_last_error(GCONV_ERR_INVALID_ARG, "bytes pointer is NULL");
  *bytes = scan_bwd_workspace_bytes(q.B, q.T, q.D);
  return GCONV_OK;
}

gconv_status gconv_gated_scan_bwd(const void* dy, const float* dhT, const void* x, const void* r, const void* i,
                                  const float* lam, const int32_t* lens, const void* saved, void* dx, void* dr,
                                  void* di, float* dlam, float* dh0, const gconv_scan_problem* p, gconv_dtype dt,
                                  void* workspace, int64_t workspace_bytes, struct CUstream_st* stream) {
  ScanArgs q;
  gconv_status s = check_scan(p, dt, &q);
  if (s != GCONV_OK) return s;
  if (dy == nullptr || x == nullptr || r == nullptr || i == nullptr || lam == nullptr || saved == nullptr ||
      dx == nullptr || dr == nullptr || di == nullptr || dlam == nullptr)
    return set_last_error(GCONV_ERR_INVALID_ARG, "dy, x, r, i, lam, saved, dx, dr, di and dlam must not be NULL");
  if (reinterpret_cast<uintptr_t>(saved) & 15)
    return set_last_error(GCONV_ERR_INVALID_ARG, "saved must be 16-byte aligned");
  const int64_t need = scan_bwd_workspace_bytes(q.B, q.T, q.D);
  s = check_workspace(workspace, workspace_bytes, need);
  if (s != GCONV_OK) return s;
  const int es = dtype_bytes((DType)dt);
  const int64_t hb = q.B * (int64_t)q.D * 4;
  if (clash({strided(dx, q.B, q.T, q.D, q.sx, es), strided(dr, q.B, q.T, q.D, q.sr, es),
             strided(di, q.B, q.T, q.D, q.si, es), packed(dlam, (int64_t)q.D * 4), packed(dh0, hb),
             packed(workspace, need)},
            {strided(x, q.B, q.T, q.D, q.sx, es), strided(r, q.B, q.T, q.D, q.sr, es),
             strided(i, q.B, q.T, q.D, q.si, es), strided(dy, q.B, q.T, q.D, q.sy, es), packed(dhT, hb),
             packed(lam, (int64_t)q.D * 4), packed(saved, scan_saved_bytes(q.B, q.T, q.D)), packed(lens, q.B * 4)}))
    return set_last_error(GCONV_ERR_INVALID_ARG, "an output or the workspace overlaps another buffer");
  LaunchArgs a;
  DeviceInfo dev;
  s = prepare(stream, dt, &a, &dev);
  if (s != GCONV_OK) return s;
  q.dy = dy, q.dhT = dhT, q.x = x, q.r = r, q.i = i, q.lam = lam, q.lens = lens;
  q.saved = static_cast<float*>(const_cast<void*>(saved));
  q.dx = dx, q.dr = dr, q.di = di, q.dlam = dlam, q.dh0 = dh0, q.ws = static_cast<float*>(workspace);
  return done(scan_bwd_launch(q, a, dev));
}

gconv_status gconv_rms_norm_q8(const void* x, const void* residual, const void* weight, void* residual_out, void* y,
                               int8_t* q, float* scale, const gconv_norm_problem* p, gconv_dtype dt,
                               struct CUstream_st* stream) {
  NormArgs n;
  gconv_status s = check_norm(p, dt, &n);
  if (s != GCONV_OK) return s;
  if ((q == nullptr) != (scale == nullptr))
    return set_last_error(GCONV_ERR_INVALID_ARG, "q and scale must be given together");
  if (y == nullptr && q == nullptr) return set_last_error(GCONV_ERR_INVALID_ARG, "y and q are both NULL");
  if (n.rows == 0) return GCONV_OK;
  if (x == nullptr) return set_last_error(GCONV_ERR_INVALID_ARG, "x must not be NULL");
  const int es = dtype_bytes((DType)dt);
  const Span xs = strided(x, 1, n.rows, n.D, {n.rows * n.sx, n.sx}, es);
  const Span rs = strided(residual, 1, n.rows, n.D, {n.rows * n.sr, n.sr}, es);
  const Span os = strided(residual_out, 1, n.rows, n.D, {n.rows * n.sr, n.sr}, es);
  const Span ys = strided(y, 1, n.rows, n.D, {n.rows * n.sy, n.sy}, es);
  const Span qs = packed(q, n.rows * n.D), ss = packed(scale, n.rows * 4), ws = packed(weight, (int64_t)n.D * es);
  // residual_out may be x or residual: the same element is read, then written, by the same thread.
  const bool same_x = residual_out == x && n.sr == n.sx, same_r = residual_out == residual;
  if (clash({os, ys, qs, ss}, {ws}) || clash({ys, qs, ss}, {xs, rs}) || (!same_x && touch(os, xs)) ||
      (!same_r && touch(os, rs)))
    return set_last_error(GCONV_ERR_INVALID_ARG, "an output overlaps an input or another output");
  LaunchArgs a;
  DeviceInfo dev;
  s = prepare(stream, dt, &a, &dev);
  if (s != GCONV_OK) return s;
  n.x = x, n.res = residual, n.w = weight, n.res_out = residual_out, n.y = y, n.q = q, n.scale = scale, n.norm = true;
  return done(norm_q8_launch(n, a, dev));
}

gconv_status gconv_quantize_rows_q8(const void* x, int8_t* q, float* scale, const gconv_norm_problem* p, gconv_dtype dt,
                                    struct CUstream_st* stream) {
  NormArgs n;
  gconv_status s = check_norm(p, dt, &n);
  if (s != GCONV_OK) return s;
  if (n.rows == 0) return GCONV_OK;
  if (x == nullptr || q == nullptr || scale == nullptr)
    return set_last_error(GCONV_ERR_INVALID_ARG, "x, q and scale must not be NULL");
  const Span xs = strided(x, 1, n.rows, n.D, {n.rows * n.sx, n.sx}, dtype_bytes((DType)dt));
  if (clash({packed(q, n.rows * n.D), packed(scale, n.rows * 4)}, {xs}))
    return set_last_error(GCONV_ERR_INVALID_ARG, "an output overlaps an input or another output");
  LaunchArgs a;
  DeviceInfo dev;
  s = prepare(stream, dt, &a, &dev);
  if (s != GCONV_OK) return s;
  n.x = x, n.q = q, n.scale = scale, n.norm = false;
  return done(norm_q8_launch(n, a, dev));
}

gconv_status gconv_matmul_q8(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                             const void* bias, void* y, const gconv_matmul_q8_problem* p, gconv_dtype dt,
                             struct CUstream_st* stream) {
  if (p == nullptr) return set_last_error(GCONV_ERR_INVALID_ARG, "problem pointer is NULL");
  if (p->reserved != 0) return set_last_error(GCONV_ERR_INVALID_ARG, "reserved field must be 0");
  if (p->M < 0 || p->M > 0x7fffffff || p->N < 1 || p->N > GCONV_MATMUL_Q8_MAX_N)
    return set_last_error(GCONV_ERR_INVALID_ARG, "M must be 0 ... 2^31 - 1 and N 1 ... %d", GCONV_MATMUL_Q8_MAX_N);
  if (p->K < 1 || p->K > GCONV_MATMUL_Q8_MAX_K)
    return set_last_error(GCONV_ERR_INVALID_ARG, "K must be 1 ... %d", GCONV_MATMUL_Q8_MAX_K);
  if (p->y_stride != 0 && (p->y_stride < p->N || (double)p->M * (double)p->y_stride > 1e18))
    return set_last_error(GCONV_ERR_INVALID_ARG, "y_stride is below N or out of range");
  gconv_status s = check_dtype(dt);
  if (s != GCONV_OK) return s;
  if (p->M == 0) return GCONV_OK;
  if (xq == nullptr || x_scale == nullptr || wq == nullptr || w_scale == nullptr || y == nullptr)
    return set_last_error(GCONV_ERR_INVALID_ARG, "xq, x_scale, wq, w_scale and y must not be NULL");
  MatmulQ8Args m;
  m.M = p->M, m.N = p->N, m.K = p->K, m.ys = p->y_stride ? p->y_stride : p->N;
  const int es = dtype_bytes((DType)dt);
  if (clash({strided(y, 1, m.M, m.N, {m.M * m.ys, m.ys}, es)},
            {packed(xq, m.M * m.K), packed(x_scale, m.M * 4), packed(wq, (int64_t)m.N * m.K),
             packed(w_scale, (int64_t)m.N * 4), packed(bias, (int64_t)m.N * es)}))
    return set_last_error(GCONV_ERR_INVALID_ARG, "y overlaps an input");
  LaunchArgs a;
  DeviceInfo dev;
  s = prepare(stream, dt, &a, &dev);
  if (s != GCONV_OK) return s;
  m.xq = xq, m.sx = x_scale, m.wq = wq, m.sw = w_scale, m.bias = bias, m.y = y;
  return done(matmul_q8_launch(m, a, dev));
}

}  // extern "C"
