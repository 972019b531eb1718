// C ABI of the token-mixer operators (include/ttt.h): argument checks, workspace planning and
// the enqueue order of short_conv.cu, head_norm.cu and selective_scan.cu.
#include <climits>

#include "api_common.h"
#include "mixer.h"

namespace ttt {
namespace {

int dtype_tag(int32_t dtype) { return dtype == TTT_DTYPE_BF16 ? DT_BF16 : DT_F32; }

ttt_status check_dtype(int32_t dtype) {
  if (dtype != TTT_DTYPE_FP32 && dtype != TTT_DTYPE_BF16)
    return fail(TTT_ERR_INVALID_ARG, "dtype must be TTT_DTYPE_FP32 or TTT_DTYPE_BF16");
  return TTT_OK;
}

// A buffer of a call: `elems` elements of `size` bytes (its whole extent, strides included).
struct Buf {
  const char* name;
  const void* p;
  long long elems;
  int size;
};

// Element alignment of every buffer, and no output on top of an input or another output.
ttt_status check_buffers(std::initializer_list<Buf> ins, std::initializer_list<Buf> outs) {
  for (const auto* list : {&ins, &outs})
    for (const Buf& x : *list)
      if (reinterpret_cast<uintptr_t>(x.p) % x.size)
        return fail(TTT_ERR_INVALID_ARG, "%s must be aligned to its %d-byte elements", x.name, x.size);
  auto meet = [](const Buf& x, const Buf& y) {
    const char* a = static_cast<const char*>(x.p);
    const char* b = static_cast<const char*>(y.p);
    return a && b && x.elems > 0 && y.elems > 0 && a < b + y.elems * y.size && b < a + x.elems * x.size;
  };
  for (const Buf* o = outs.begin(); o != outs.end(); ++o) {
    for (const Buf& x : ins)
      if (meet(x, *o)) return fail(TTT_ERR_INVALID_ARG, "%s overlaps %s", o->name, x.name);
    for (const Buf* q = outs.begin(); q != o; ++q)
      if (meet(*q, *o)) return fail(TTT_ERR_INVALID_ARG, "%s overlaps %s", o->name, q->name);
  }
  return TTT_OK;
}

// Elements that `rows` rows of `width` elements, `stride` apart, span.
long long extent(long long rows, long long stride, long long width) {
  return rows > 0 ? (rows - 1) * stride + width : 0;
}

// A row stride of the descriptor: 0 means dense.
ttt_status resolve_row(const char* name, int64_t row, long long width, long long* out) {
  if (row != 0 && (row < width || row > (1LL << 31)))
    return fail(TTT_ERR_INVALID_ARG, "%s must be 0 (dense) or in %lld..2^31", name, width);
  *out = row ? row : width;
  return TTT_OK;
}

ttt_status check_tokens(int32_t B, int32_t N) {
  if (B < 0 || N < 0) return fail(TTT_ERR_INVALID_ARG, "B and N must be >= 0");
  if (B > 65535) return fail(TTT_ERR_UNSUPPORTED, "B must be <= 65535");
  if (N > (1 << 22)) return fail(TTT_ERR_UNSUPPORTED, "N must be <= 4194304");
  if ((long long)B * N > INT_MAX) return fail(TTT_ERR_UNSUPPORTED, "B*N must be < 2^31");
  return TTT_OK;
}

// ------------------------------------------------------------------ short convolution
ttt_status check_conv(const ttt_conv_desc* d, bool step, ConvArgs* a) {
  if (!d) return fail(TTT_ERR_INVALID_ARG, "desc is NULL");
  TTT_TRY(check_tokens(d->B, d->N));
  if (d->D < 1) return fail(TTT_ERR_INVALID_ARG, "D must be >= 1");
  TTT_TRY(check_dtype(d->dtype));
  if (d->act != TTT_ACT_NONE && d->act != TTT_ACT_SILU)
    return fail(TTT_ERR_INVALID_ARG, "act must be TTT_ACT_NONE or TTT_ACT_SILU");
  if (d->width < 1) return fail(TTT_ERR_INVALID_ARG, "width must be >= 1");
  if (d->width < 2 || d->width > 8) return fail(TTT_ERR_UNSUPPORTED, "width must be in 2..8");
  if (d->D > (1 << 20)) return fail(TTT_ERR_UNSUPPORTED, "D must be <= 1048576");
  if (step && d->N != 1) return fail(TTT_ERR_INVALID_ARG, "a step takes N = 1");
  *a = ConvArgs{};
  a->B = d->B; a->N = d->N; a->D = d->D; a->width = d->width; a->act = d->act == TTT_ACT_SILU;
  return resolve_row("x_row", d->x_row, d->D, &a->x_row);
}

size_t plan_conv(const ConvArgs& a, void* base, float** partials) {
  Carve cv(base);
  *partials = cv.take_n<float>(conv_bwd_rows(a.B, a.N, a.D) * (a.width + 1) * a.D);
  return cv.off;
}

// ------------------------------------------------------------------ heads
ttt_status check_heads(const ttt_heads_desc* d, HeadArgs* a) {
  if (!d) return fail(TTT_ERR_INVALID_ARG, "desc is NULL");
  TTT_TRY(check_tokens(d->B, d->N));
  if (d->h < 1) return fail(TTT_ERR_INVALID_ARG, "h must be >= 1");
  if (d->Hq < 0 || d->Hk < 0 || d->Hv < 0)
    return fail(TTT_ERR_INVALID_ARG, "Hq, Hk and Hv must be >= 0");
  TTT_TRY(check_dtype(d->dtype));
  if (d->norm != TTT_NORM_NONE && d->norm != TTT_NORM_RMS && d->norm != TTT_NORM_L2)
    return fail(TTT_ERR_INVALID_ARG, "norm must be one of TTT_NORM_*");
  if (d->pairs != TTT_PAIRS_HALVES && d->pairs != TTT_PAIRS_INTERLEAVED)
    return fail(TTT_ERR_INVALID_ARG, "pairs must be one of TTT_PAIRS_*");
  if (d->rot < 0 || d->rot > d->h || d->rot % 2)
    return fail(TTT_ERR_INVALID_ARG, "rot must be even and in 0..h");
  if (!(d->eps >= 0.0f) || (d->norm != TTT_NORM_NONE && !(d->eps > 0.0f)))
    return fail(TTT_ERR_INVALID_ARG, "eps must be > 0 with a norm (a zero row has no direction)");
  if (d->h > 512) return fail(TTT_ERR_UNSUPPORTED, "h must be <= 512");
  if (d->Hq > 65535 || d->Hk > 65535 || d->Hv > 65535)
    return fail(TTT_ERR_UNSUPPORTED, "Hq, Hk and Hv must be <= 65535");
  if (d->pos0 < 0) return fail(TTT_ERR_INVALID_ARG, "pos0 must be >= 0");
  *a = HeadArgs{};
  a->B = d->B; a->N = d->N; a->h = d->h; a->norm = d->norm; a->rot = d->rot; a->pairs = d->pairs;
  a->eps = d->eps; a->pos0 = d->pos0;
  a->H[0] = d->Hq; a->H[1] = d->Hk; a->H[2] = d->Hv;
  TTT_TRY(resolve_row("q_row", d->q_row, (long long)d->Hq * d->h, &a->row[0]));
  TTT_TRY(resolve_row("k_row", d->k_row, (long long)d->Hk * d->h, &a->row[1]));
  return resolve_row("v_row", d->v_row, (long long)d->Hv * d->h, &a->row[2]);
}

size_t plan_heads(const HeadArgs& a, void* base, float** partials) {
  Carve cv(base);
  *partials = cv.take_n<float>(head_bwd_max_rows(a.B, a.N) * 2 * a.h);
  return cv.off;
}

// ------------------------------------------------------------------ selective scan
ttt_status check_scan(const ttt_scan_desc* d, bool step, ScanArgs* a) {
  if (!d) return fail(TTT_ERR_INVALID_ARG, "desc is NULL");
  TTT_TRY(check_tokens(d->B, d->N));
  if (d->D < 1 || d->S < 1 || d->G < 1) return fail(TTT_ERR_INVALID_ARG, "D, S and G must be >= 1");
  TTT_TRY(check_dtype(d->dtype));
  if (d->D % d->G) return fail(TTT_ERR_INVALID_ARG, "D must be a multiple of G");
  if (d->softplus != 0 && d->softplus != 1) return fail(TTT_ERR_INVALID_ARG, "softplus must be 0 or 1");
  if (d->reserved != 0) return fail(TTT_ERR_INVALID_ARG, "reserved must be 0");
  if (d->S > kScanMaxState) return fail(TTT_ERR_UNSUPPORTED, "S must be <= %d", kScanMaxState);
  if (d->D > (1 << 20)) return fail(TTT_ERR_UNSUPPORTED, "D must be <= 1048576");
  if ((long long)d->B * d->D > INT_MAX) return fail(TTT_ERR_UNSUPPORTED, "B*D must be < 2^31");
  if (step && d->N != 1) return fail(TTT_ERR_INVALID_ARG, "a step takes N = 1");
  *a = ScanArgs{};
  a->B = d->B; a->N = d->N; a->D = d->D; a->S = d->S; a->G = d->G; a->softplus = d->softplus;
  TTT_TRY(resolve_row("u_row", d->u_row, d->D, &a->u_row));
  TTT_TRY(resolve_row("dt_row", d->dt_row, d->D, &a->dt_row));
  TTT_TRY(resolve_row("z_row", d->z_row, d->D, &a->z_row));
  TTT_TRY(resolve_row("b_row", d->b_row, (long long)d->G * d->S, &a->b_row));
  return resolve_row("c_row", d->c_row, (long long)d->G * d->S, &a->c_row);
}

size_t plan_scan_fwd(ScanArgs& a, void* base) {
  Carve cv(base);
  a.chunks = scan_chunks(a.B, a.N, a.D, a.G, a.S, false, &a.chunk);
  if (a.chunks == 1) return 0;   // one pass, straight from state_in
  const long long bk = (long long)a.B * a.chunks;
  a.ends = cv.take_n<float>(bk * a.D * scan_padded_state(a.S));
  a.dsum = cv.take_n<float>(bk * a.D);
  return cv.off;
}

size_t plan_scan_bwd(ScanArgs& a, void* base) {
  Carve cv(base);
  a.chunks = scan_chunks(a.B, a.N, a.D, a.G, a.S, true, &a.chunk);
  const long long SP = scan_padded_state(a.S), bk = (long long)a.B * a.chunks;
  const long long subs = (long long)a.B * ((a.N + kScanSub - 1) / kScanSub);
  a.ends = cv.take_n<float>(bk * a.D * SP);
  a.dsum = cv.take_n<float>(bk * a.D);
  a.back = cv.take_n<float>(bk * a.D * SP);
  a.marks = cv.take_n<float>(subs * a.D * SP);
  a.msum = cv.take_n<float>(subs * a.D);
  a.bcpart = cv.take_n<float>((long long)scan_channel_blocks(a.D, a.G, a.S) * a.B * a.N * a.G * 2 * SP);
  a.part = cv.take_n<float>(bk * a.D * (a.S + 2));
  return cv.off;
}

}  // namespace
}  // namespace ttt

using namespace ttt;

extern "C" {

// ------------------------------------------------------------------ short convolution
ttt_status ttt_short_conv_fwd(const ttt_conv_desc* desc, const void* x, const float* w,
                              const float* bias, const void* state_in, const int32_t* lens, void* y,
                              void* state_out, ttt_stream_t stream) {
  ConvArgs a;
  TTT_TRY(check_conv(desc, false, &a));
  if (a.B == 0) return TTT_OK;
  if (!w) return fail(TTT_ERR_INVALID_ARG, "w must not be NULL");
  if (a.N > 0 && (!x || !y)) return fail(TTT_ERR_INVALID_ARG, "x and y must not be NULL");
  const long long rows = (long long)a.B * a.N, st = (long long)a.B * (a.width - 1) * a.D;
  const int dt = dtype_tag(desc->dtype), size = (int)dtype_size(dt);
  const Buf out_state = {"state_out", state_out, st, size};
  TTT_TRY(check_buffers({{"x", x, extent(rows, a.x_row, a.D), size},
                         {"w", w, (long long)a.width * a.D, 4},
                         {"bias", bias, a.D, 4},
                         {"lens", lens, a.B, 4},
                         {"state_in", state_in, state_in == state_out ? 0 : st, size}},
                        {{"y", y, rows * a.D, size}, out_state}));
  a.x = x; a.w = w; a.bias = bias; a.state_in = state_in; a.lens = lens; a.y = y;
  a.state_out = state_out;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.N == 0 && !state_out) return TTT_OK;
  t_guards.clear();
  return with_checks(s, {{y, rows * a.D, dt}, {state_out, st, dt}}, [&]() -> ttt_status {
    TTT_OP("short_conv", conv_fwd(dt, a, s));
    return TTT_OK;
  });
}

ttt_status ttt_short_conv_step(const ttt_conv_desc* desc, const void* x, const float* w,
                               const float* bias, void* state, void* y, ttt_stream_t stream) {
  ConvArgs a;
  TTT_TRY(check_conv(desc, true, &a));
  if (a.B == 0) return TTT_OK;
  if (!x || !w || !state || !y)
    return fail(TTT_ERR_INVALID_ARG, "x, w, state and y must not be NULL");
  const long long st = (long long)a.B * (a.width - 1) * a.D, n = (long long)a.B * a.D;
  const int dt = dtype_tag(desc->dtype), size = (int)dtype_size(dt);
  TTT_TRY(check_buffers({{"x", x, extent(a.B, a.x_row, a.D), size},
                         {"w", w, (long long)a.width * a.D, 4},
                         {"bias", bias, a.D, 4}},
                        {{"state", state, st, size}, {"y", y, n, size}}));
  a.x = x; a.w = w; a.bias = bias; a.state_out = state; a.y = y;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  t_guards.clear();
  return with_checks(s, {{y, n, dt}, {state, st, dt}}, [&]() -> ttt_status {
    TTT_OP("short_conv_step", conv_step(dt, a, s));
    return TTT_OK;
  });
}

size_t ttt_short_conv_bwd_workspace_bytes(const ttt_conv_desc* desc) {
  ConvArgs a;
  if (check_conv(desc, false, &a) != TTT_OK) return 0;
  float* p;
  return plan_conv(a, nullptr, &p);
}

ttt_status ttt_short_conv_bwd(const ttt_conv_desc* desc, const void* x, const float* w,
                              const float* bias, const void* state_in, const int32_t* lens,
                              const void* dy, const void* dstate_out, void* dx, float* dw,
                              float* dbias, void* dstate_in, void* workspace,
                              size_t workspace_bytes, ttt_stream_t stream) {
  ConvArgs a;
  TTT_TRY(check_conv(desc, false, &a));
  if (!w || !dw) return fail(TTT_ERR_INVALID_ARG, "w and dw must not be NULL");
  const long long rows = (long long)a.B * a.N, st = (long long)a.B * (a.width - 1) * a.D;
  if (rows > 0 && (!x || !dy || !dx))
    return fail(TTT_ERR_INVALID_ARG, "x, dy and dx must not be NULL");
  const int dt = dtype_tag(desc->dtype), size = (int)dtype_size(dt);
  const long long taps = (long long)a.width * a.D;
  TTT_TRY(check_buffers({{"x", x, extent(rows, a.x_row, a.D), size},
                         {"w", w, taps, 4},
                         {"bias", bias, a.D, 4},
                         {"lens", lens, a.B, 4},
                         {"state_in", state_in, st, size},
                         {"dy", dy, rows * a.D, size},
                         {"dstate_out", dstate_out, st, size}},
                        {{"dx", dx, rows * a.D, size},
                         {"dw", dw, taps, 4},
                         {"dbias", dbias, a.D, 4},
                         {"dstate_in", dstate_in, st, size},
                         {"workspace", workspace, (long long)workspace_bytes, 1}}));
  float* part = nullptr;
  TTT_TRY(check_ws(workspace, workspace_bytes, plan_conv(a, nullptr, &part)));
  t_guards.clear();
  plan_conv(a, workspace, &part);
  a.x = x; a.w = w; a.bias = bias; a.state_in = state_in; a.lens = lens;
  a.dy = dy; a.dstate_out = dstate_out; a.dx = dx; a.dstate_in = dstate_in; a.partials = part;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return with_checks(s, {{dx, rows * a.D, dt}, {dw, taps, DT_F32}, {dbias, a.D, DT_F32},
                         {dstate_in, st, dt}}, [&]() -> ttt_status {
    if (a.B > 0) TTT_OP("short_conv_bwd", conv_bwd(dt, a, s));
    TTT_OP("short_conv_bwd_sum",
           column_sums(part, conv_bwd_rows(a.B, a.N, a.D), {{dw, dbias, nullptr}, {taps, a.D, 0}}, s));
    return TTT_OK;
  });
}

// ------------------------------------------------------------------ heads
ttt_status ttt_head_norm_rope_fwd(const ttt_heads_desc* desc, const void* q, const void* k,
                                  const void* v, const float* wq, const float* wk,
                                  const float* inv_freq, const int32_t* positions, void* q_out,
                                  void* k_out, void* v_out, ttt_stream_t stream) {
  HeadArgs a;
  TTT_TRY(check_heads(desc, &a));
  const long long M = (long long)a.B * a.N;
  if (M == 0 || a.H[0] + a.H[1] + a.H[2] == 0) return TTT_OK;
  const void* x[3] = {q, k, v};
  void* out[3] = {q_out, k_out, v_out};
  for (int i = 0; i < 3; ++i)
    if (a.H[i] && (!x[i] || !out[i]))
      return fail(TTT_ERR_INVALID_ARG, "a tensor with heads needs its input and output");
  if (a.rot && !inv_freq) return fail(TTT_ERR_INVALID_ARG, "rot > 0 needs inv_freq");
  const int dt = dtype_tag(desc->dtype), size = (int)dtype_size(dt);
  long long in[3], n[3];
  for (int i = 0; i < 3; ++i) {
    n[i] = M * a.H[i] * a.h;
    in[i] = a.H[i] ? extent(M, a.row[i], (long long)a.H[i] * a.h) : 0;
    a.x[i] = x[i];
    a.out[i] = out[i];
  }
  TTT_TRY(check_buffers({{"q", q, in[0], size}, {"k", k, in[1], size}, {"v", v, in[2], size},
                         {"wq", wq, a.h, 4}, {"wk", wk, a.h, 4}, {"inv_freq", inv_freq, a.rot / 2, 4},
                         {"positions", positions, M, 4}},
                        {{"q_out", q_out, n[0], size}, {"k_out", k_out, n[1], size},
                         {"v_out", v_out, n[2], size}}));
  a.w[0] = wq; a.w[1] = wk; a.inv_freq = inv_freq; a.positions = positions;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  t_guards.clear();
  return with_checks(s, {{q_out, n[0], dt}, {k_out, n[1], dt}, {v_out, n[2], dt}},
                     [&]() -> ttt_status {
    TTT_OP("head_norm_rope", head_fwd(dt, a, s));
    return TTT_OK;
  });
}

size_t ttt_head_norm_rope_bwd_workspace_bytes(const ttt_heads_desc* desc) {
  HeadArgs a;
  if (check_heads(desc, &a) != TTT_OK) return 0;
  float* p;
  return plan_heads(a, nullptr, &p);
}

ttt_status ttt_head_norm_rope_bwd(const ttt_heads_desc* desc, const void* q, const void* k,
                                  const float* wq, const float* wk, const float* inv_freq,
                                  const int32_t* positions, const void* dq_out,
                                  const void* dk_out, const void* dv_out, void* dq, void* dk,
                                  void* dv, float* dwq, float* dwk, void* workspace,
                                  size_t workspace_bytes, ttt_stream_t stream) {
  HeadArgs a;
  TTT_TRY(check_heads(desc, &a));
  const long long M = (long long)a.B * a.N;
  const void* x[3] = {q, k, nullptr};
  const void* dout[3] = {dq_out, dk_out, dv_out};
  void* dx[3] = {dq, dk, dv};
  if ((dwq && !wq) || (dwk && !wk))
    return fail(TTT_ERR_INVALID_ARG, "a weight gradient needs its weight");
  const int dt = dtype_tag(desc->dtype), size = (int)dtype_size(dt);
  long long in[3], n[3];
  for (int i = 0; i < 3; ++i) {
    if (M > 0 && a.H[i] && ((i < 2 && !x[i]) || !dout[i] || !dx[i]))
      return fail(TTT_ERR_INVALID_ARG, "a tensor with heads needs its input and both gradients");
    n[i] = M * a.H[i] * a.h;
    in[i] = a.H[i] && x[i] ? extent(M, a.row[i], (long long)a.H[i] * a.h) : 0;
    a.x[i] = x[i];
    a.dout[i] = dout[i];
    a.dx[i] = dx[i];
  }
  if (M > 0 && a.rot && !inv_freq) return fail(TTT_ERR_INVALID_ARG, "rot > 0 needs inv_freq");
  TTT_TRY(check_buffers({{"q", q, in[0], size}, {"k", k, in[1], size}, {"wq", wq, a.h, 4},
                         {"wk", wk, a.h, 4}, {"inv_freq", inv_freq, a.rot / 2, 4},
                         {"positions", positions, M, 4}, {"dq_out", dq_out, n[0], size},
                         {"dk_out", dk_out, n[1], size}, {"dv_out", dv_out, n[2], size}},
                        {{"dq", dq, n[0], size}, {"dk", dk, n[1], size}, {"dv", dv, n[2], size},
                         {"dwq", dwq, a.h, 4}, {"dwk", dwk, a.h, 4},
                         {"workspace", workspace, (long long)workspace_bytes, 1}}));
  const bool sums = dwq || dwk;
  float* part = nullptr;
  t_guards.clear();
  if (sums) {
    TTT_TRY(check_ws(workspace, workspace_bytes, plan_heads(a, nullptr, &part)));
    t_guards.clear();
    plan_heads(a, workspace, &part);
  }
  a.w[0] = wq; a.w[1] = wk; a.inv_freq = inv_freq; a.positions = positions; a.partials = part;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return with_checks(s, {{dq, n[0], dt}, {dk, n[1], dt}, {dv, n[2], dt},
                         {dwq, a.h, DT_F32}, {dwk, a.h, DT_F32}}, [&]() -> ttt_status {
    const bool any = M > 0 && a.H[0] + a.H[1] + a.H[2] > 0;
    long long rows = 0;
    if (any) TTT_OP("head_norm_rope_bwd", head_bwd(dt, a, &rows, s));
    if (sums)
      TTT_OP("head_norm_rope_bwd_sum",
             column_sums(part, rows, {{dwq, dwk, nullptr}, {a.h, a.h, 0}}, s));
    return TTT_OK;
  });
}

// ------------------------------------------------------------------ selective scan
size_t ttt_selective_scan_workspace_bytes(const ttt_scan_desc* desc, int32_t backward) {
  ScanArgs a;
  if (check_scan(desc, false, &a) != TTT_OK) return 0;
  return backward ? plan_scan_bwd(a, nullptr) : plan_scan_fwd(a, nullptr);
}

ttt_status ttt_selective_scan_fwd(const ttt_scan_desc* desc, const void* u, const void* dt,
                                  const float* A, const void* Bm, const void* Cm, const float* D,
                                  const void* z, const float* dt_bias, const float* state_in,
                                  const int32_t* lens, void* y, float* state_out, void* workspace,
                                  size_t workspace_bytes, ttt_stream_t stream) {
  ScanArgs a;
  TTT_TRY(check_scan(desc, false, &a));
  if (a.B == 0) return TTT_OK;
  if (!A) return fail(TTT_ERR_INVALID_ARG, "A must not be NULL");
  if (a.N > 0 && (!u || !dt || !Bm || !Cm || !y))
    return fail(TTT_ERR_INVALID_ARG, "u, dt, Bm, Cm and y must not be NULL");
  const long long rows = (long long)a.B * a.N, st = (long long)a.B * a.D * a.S;
  const long long gs = (long long)a.G * a.S;
  const int tag = dtype_tag(desc->dtype), size = (int)dtype_size(tag);
  const size_t need = plan_scan_fwd(a, nullptr);
  // The first pass of a split sequence and the join read state_in before the outputs pass
  // writes state_out, and an unsplit pass reads and writes each element in one thread.
  TTT_TRY(check_buffers({{"u", u, extent(rows, a.u_row, a.D), size},
                         {"dt", dt, extent(rows, a.dt_row, a.D), size},
                         {"A", A, (long long)a.D * a.S, 4},
                         {"Bm", Bm, extent(rows, a.b_row, gs), size},
                         {"Cm", Cm, extent(rows, a.c_row, gs), size},
                         {"D", D, a.D, 4},
                         {"z", z, extent(rows, a.z_row, a.D), size},
                         {"dt_bias", dt_bias, a.D, 4},
                         {"state_in", state_in, state_in == state_out ? 0 : st, 4},
                         {"lens", lens, a.B, 4}},
                        {{"y", y, rows * a.D, size},
                         {"state_out", state_out, st, 4},
                         {"workspace", workspace, need ? (long long)workspace_bytes : 0, 1}}));
  TTT_TRY(check_ws(workspace, workspace_bytes, need));
  t_guards.clear();
  plan_scan_fwd(a, need ? workspace : nullptr);
  a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = D; a.z = z; a.dt_bias = dt_bias;
  a.state_in = state_in; a.lens = lens; a.y = y; a.state_out = state_out;
  if (a.N == 0 && !state_out) return TTT_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return with_checks(s, {{y, rows * a.D, tag}, {state_out, st, DT_F32}}, [&]() -> ttt_status {
    if (a.chunks > 1) {
      TTT_OP("selective_scan_ends", scan_fwd_ends(tag, a, s));
      TTT_OP("selective_scan_join", scan_join(a, false, s));
    }
    TTT_OP("selective_scan", scan_fwd_outputs(tag, a, s));
    return TTT_OK;
  });
}

ttt_status ttt_selective_scan_step(const ttt_scan_desc* desc, const void* u, const void* dt,
                                   const float* A, const void* Bm, const void* Cm, const float* D,
                                   const void* z, const float* dt_bias, float* state, void* y,
                                   ttt_stream_t stream) {
  ScanArgs a;
  TTT_TRY(check_scan(desc, true, &a));
  if (a.B == 0) return TTT_OK;
  if (!u || !dt || !A || !Bm || !Cm || !state || !y)
    return fail(TTT_ERR_INVALID_ARG, "u, dt, A, Bm, Cm, state and y must not be NULL");
  const long long n = (long long)a.B * a.D, st = n * a.S, gs = (long long)a.G * a.S;
  const int tag = dtype_tag(desc->dtype), size = (int)dtype_size(tag);
  TTT_TRY(check_buffers({{"u", u, extent(a.B, a.u_row, a.D), size},
                         {"dt", dt, extent(a.B, a.dt_row, a.D), size},
                         {"A", A, (long long)a.D * a.S, 4},
                         {"Bm", Bm, extent(a.B, a.b_row, gs), size},
                         {"Cm", Cm, extent(a.B, a.c_row, gs), size},
                         {"D", D, a.D, 4},
                         {"z", z, extent(a.B, a.z_row, a.D), size},
                         {"dt_bias", dt_bias, a.D, 4}},
                        {{"state", state, st, 4}, {"y", y, n, size}}));
  a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = D; a.z = z; a.dt_bias = dt_bias;
  a.state_out = state; a.y = y;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  t_guards.clear();
  return with_checks(s, {{y, n, tag}, {state, st, DT_F32}}, [&]() -> ttt_status {
    TTT_OP("selective_scan_step", scan_step(tag, a, s));
    return TTT_OK;
  });
}

ttt_status ttt_selective_scan_bwd(const ttt_scan_desc* desc, const void* u, const void* dt,
                                  const float* A, const void* Bm, const void* Cm, const float* D,
                                  const void* z, const float* dt_bias, const float* state_in,
                                  const int32_t* lens, const void* dy, const float* dstate_out,
                                  void* du, void* ddt, float* dA, void* dBm, void* dCm, float* dD,
                                  void* dz, float* ddt_bias, float* dstate_in, void* workspace,
                                  size_t workspace_bytes, ttt_stream_t stream) {
  ScanArgs a;
  TTT_TRY(check_scan(desc, false, &a));
  if (!A || !dA) return fail(TTT_ERR_INVALID_ARG, "A and dA must not be NULL");
  const long long rows = (long long)a.B * a.N, st = (long long)a.B * a.D * a.S;
  const long long gs = (long long)a.G * a.S;
  if (rows > 0 && (!u || !dt || !Bm || !Cm || !dy || !du || !ddt || !dBm || !dCm))
    return fail(TTT_ERR_INVALID_ARG, "u, dt, Bm, Cm, dy, du, ddt, dBm and dCm must not be NULL");
  if (rows > 0 && (z != nullptr) != (dz != nullptr))
    return fail(TTT_ERR_INVALID_ARG, "z and dz go together");
  const int tag = dtype_tag(desc->dtype), size = (int)dtype_size(tag);
  TTT_TRY(check_buffers({{"u", u, extent(rows, a.u_row, a.D), size},
                         {"dt", dt, extent(rows, a.dt_row, a.D), size},
                         {"A", A, (long long)a.D * a.S, 4},
                         {"Bm", Bm, extent(rows, a.b_row, gs), size},
                         {"Cm", Cm, extent(rows, a.c_row, gs), size},
                         {"D", D, a.D, 4},
                         {"z", z, extent(rows, a.z_row, a.D), size},
                         {"dt_bias", dt_bias, a.D, 4},
                         {"state_in", state_in, st, 4},
                         {"lens", lens, a.B, 4},
                         {"dy", dy, rows * a.D, size},
                         {"dstate_out", dstate_out, st, 4}},
                        {{"du", du, rows * a.D, size},
                         {"ddt", ddt, rows * a.D, size},
                         {"dA", dA, (long long)a.D * a.S, 4},
                         {"dBm", dBm, rows * gs, size},
                         {"dCm", dCm, rows * gs, size},
                         {"dD", dD, a.D, 4},
                         {"dz", dz, rows * a.D, size},
                         {"ddt_bias", ddt_bias, a.D, 4},
                         {"dstate_in", dstate_in, st, 4},
                         {"workspace", workspace, (long long)workspace_bytes, 1}}));
  TTT_TRY(check_ws(workspace, workspace_bytes, plan_scan_bwd(a, nullptr)));
  t_guards.clear();
  plan_scan_bwd(a, workspace);
  a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = D; a.z = z; a.dt_bias = dt_bias;
  a.state_in = state_in; a.lens = lens; a.dy = dy; a.dstate_out = dstate_out;
  a.du = du; a.ddt = ddt; a.dA = dA; a.dB = dBm; a.dC = dCm; a.dD = dD; a.dz = dz;
  a.ddt_bias = ddt_bias; a.dstate_in = dstate_in;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return with_checks(s, {{du, rows * a.D, tag}, {ddt, rows * a.D, tag}, {dA, (long long)a.D * a.S, DT_F32},
                         {dBm, rows * gs, tag}, {dCm, rows * gs, tag}, {dD, a.D, DT_F32},
                         {dz, dz ? rows * a.D : 0, tag}, {ddt_bias, a.D, DT_F32},
                         {dstate_in, st, DT_F32}}, [&]() -> ttt_status {
    const long long bk = (long long)a.B * a.chunks;
    if (a.B > 0) {
      TTT_OP("selective_scan_marks", scan_bwd_marks(tag, a, s));
      if (a.chunks > 1) TTT_OP("selective_scan_join", scan_join(a, true, s));
      TTT_OP("selective_scan_bwd", scan_bwd_main(tag, a, s));
      if (a.N > 0) TTT_OP("selective_scan_sum_bc", scan_bwd_sum_bc(tag, a, s));
    }
    TTT_OP("selective_scan_sum_ad",
           column_sums(a.part, bk, {{dA, dD, ddt_bias}, {(long long)a.D * a.S, a.D, a.D}}, s));
    return TTT_OK;
  });
}

}  // extern "C"
