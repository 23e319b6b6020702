// C ABI entry points of the gated recurrence a channel, the short convolution and the norms
// around a block: argument checks and dispatch. No HIP call here; launches live in the .hip files.
#include <cmath>
#include <utility>

#include "gdn_block.h"

namespace gdn {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dtype_ok(int d) { return d == GDN_DTYPE_F32 || d == GDN_DTYPE_BF16; }

// Sizes: every element offset stays far inside int64, every grid inside 31 bits and every
// launch under 2^32 threads (at most 128 a channel of a sequence).
int sizes(int64_t B, int64_t T, int64_t C) {
  if (B < 1 || T < 0 || C < 8 || C % 8 != 0) return GDN_ERR_ARG;
  if (B > (1 << 20) || C > (1 << 16) || T > (int64_t(1) << 31) - (1 << 16)) return GDN_ERR_UNSUPPORTED;
  if (B * C > (1 << 24) || B * T > (int64_t(1) << 36)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// A token stride: 0 means contiguous; else at least a token's channels, in 16-byte steps.
int stride(int64_t given, int64_t C, int dtype, int64_t* out) {
  *out = given == 0 ? C : given;
  if (*out < C || *out % (dtype == GDN_DTYPE_BF16 ? 8 : 4) != 0) return GDN_ERR_ARG;
  if (*out > (int64_t(1) << 24)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

bool ws_ok(const void* ws, size_t bytes, size_t need) {
  return ws != nullptr && bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

// An array of T rows a sequence: NULL only where there are none.
bool rows_ok(const void* p, int64_t T) { return aligned16(p) && (T == 0 || p != nullptr); }

int64_t size_of(int dtype) { return dtype == GDN_DTYPE_BF16 ? 2 : 4; }

// Whether `bytes` from `out` on meet one of `rows` rows of `width` bytes from `in` on, `ld` >= width
// bytes apart. Absent arrays meet nothing.
bool meets(const void* out, int64_t bytes, const void* in, int64_t rows, int64_t width, int64_t ld) {
  if (out == nullptr || in == nullptr) return false;
  const int64_t at = int64_t(reinterpret_cast<uintptr_t>(out)) - int64_t(reinterpret_cast<uintptr_t>(in));
  const int64_t r = at < width ? 0 : (at - width) / ld + 1;   // the first row that ends behind out's start
  return r < rows && r * ld < at + bytes;
}

int hip_status(int rc) { return rc == 0 ? GDN_OK : GDN_ERR_HIP; }

int scan_check(const gdn_scan_args* a, ScanProblem* p) {
  if (a == nullptr || !dtype_ok(a->dtype)) return GDN_ERR_ARG;
  if (a->gate < GDN_SCAN_LOG || a->gate > GDN_SCAN_POWER) return GDN_ERR_ARG;
  int st = sizes(a->B, a->T, a->C);
  if (st != GDN_OK) return st;
  p->a = *a;
  if ((st = stride(a->x_stride, a->C, a->dtype, &p->a.x_stride)) != GDN_OK) return st;
  if ((st = stride(a->f_stride, a->C, a->dtype, &p->a.f_stride)) != GDN_OK) return st;
  return stride(a->i_stride, a->C, a->dtype, &p->a.i_stride);
}

int scan_pointers(const gdn_scan_args& a) {
  if (!rows_ok(a.x, a.T) || !rows_ok(a.f, a.T) || !aligned16(a.i) || !aligned4(a.seq_lens)) return GDN_ERR_ARG;
  // decay belongs to POWER alone
  if ((a.gate == GDN_SCAN_POWER) != (a.decay != nullptr) || !aligned16(a.decay)) return GDN_ERR_ARG;
  return GDN_OK;
}

int conv_check(const gdn_conv_args* a, ConvProblem* p) {
  if (a == nullptr || !dtype_ok(a->dtype)) return GDN_ERR_ARG;
  if (a->activation != 0 && a->activation != GDN_ACT_SILU) return GDN_ERR_ARG;
  const int st = sizes(a->B, a->T, a->C);
  if (st != GDN_OK) return st;
  if (a->W < 2 || a->W > 4) return GDN_ERR_UNSUPPORTED;
  p->a = *a;
  return stride(a->x_stride, a->C, a->dtype, &p->a.x_stride);
}

int conv_pointers(const gdn_conv_args& a) {
  if (!rows_ok(a.x, a.T) || a.w == nullptr || !aligned16(a.w) || !aligned16(a.bias) || !aligned4(a.seq_lens))
    return GDN_ERR_ARG;
  return GDN_OK;
}

int norm_check(const gdn_block_norm_args* a, BlockNormProblem* p) {
  if (a == nullptr || !dtype_ok(a->dtype)) return GDN_ERR_ARG;
  if (a->residual_dtype != GDN_DTYPE_F32 && a->residual_dtype != a->dtype) return GDN_ERR_ARG;
  if (a->activation != GDN_ACT_SILU && a->activation != GDN_ACT_SIGMOID) return GDN_ERR_ARG;
  if (a->post_norm != 0 && a->post_norm != 1) return GDN_ERR_ARG;
  if (!(a->eps >= 0.0f) || !std::isfinite(a->residual_scale)) return GDN_ERR_ARG;
  int st = sizes(a->B, a->T, a->C);
  if (st != GDN_OK) return st;
  if (a->C > 16384) return GDN_ERR_UNSUPPORTED;
  // nothing of a block without its output
  if (a->y == nullptr && a->T > 0 && (a->gate != nullptr || a->scale != nullptr || a->post_weight != nullptr || a->post_norm))
    return GDN_ERR_ARG;
  if (a->post_weight != nullptr && !a->post_norm) return GDN_ERR_ARG;
  p->a = *a;
  p->tokens = a->B * a->T;
  if ((st = stride(a->r_stride, a->C, a->residual_dtype, &p->a.r_stride)) != GDN_OK) return st;
  if ((st = stride(a->y_stride, a->C, a->dtype, &p->a.y_stride)) != GDN_OK) return st;
  return stride(a->gate_stride, a->C, a->dtype, &p->a.gate_stride);
}

int norm_pointers(const gdn_block_norm_args& a) {
  if (!rows_ok(a.r, a.T) || !aligned16(a.y) || !aligned16(a.gate)) return GDN_ERR_ARG;
  if (!aligned16(a.scale) || !aligned16(a.post_weight) || !aligned16(a.weight)) return GDN_ERR_ARG;
  return GDN_OK;
}

// y apart from x, or x itself while one thread walks a sequence's tokens in turn: else a run of tokens reads
// the rows before it after another thread may have replaced them.
bool conv_rows_apart(const gdn_conv_args& a) {
  const int64_t width = a.C * size_of(a.dtype), ld = a.x_stride * size_of(a.dtype);
  const int64_t rows = a.B * a.T;
  return !meets(a.y, rows * width, a.x, rows, width, ld) ||
         (a.y == a.x && (ld == width || rows == 1) && a.T <= kConvInPlace);
}

// out, `rows` contiguous rows of C elements, apart from in, whose rows lie ld elements from each other; or in
// itself, row over row and element over element.
bool apart_or_in_place(const void* out, int out_dtype, const void* in, int in_dtype, int64_t ld, int64_t C, int64_t rows) {
  const int64_t size = size_of(in_dtype);
  return !meets(out, rows * C * size_of(out_dtype), in, rows, C * size, ld * size) ||
         (out == in && out_dtype == in_dtype && (ld == C || rows == 1));
}
// The same for rows of the recurrence: a workgroup (or a thread) reads its own rows' channels before it
// writes them, and no other's.
bool scan_rows_apart(const gdn_scan_args& a, const void* out) {
  const int64_t rows = a.B * a.T;
  return apart_or_in_place(out, a.dtype, a.x, a.dtype, a.x_stride, a.C, rows) &&
         apart_or_in_place(out, a.dtype, a.f, a.dtype, a.f_stride, a.C, rows) &&
         apart_or_in_place(out, a.dtype, a.i, a.dtype, a.i_stride, a.C, rows);
}
bool norm_rows_apart(const gdn_block_norm_args& a, int64_t rows, const void* out, int dtype) {
  return apart_or_in_place(out, dtype, a.r, a.residual_dtype, a.r_stride, a.C, rows) &&
         apart_or_in_place(out, dtype, a.y, a.dtype, a.y_stride, a.C, rows) &&
         apart_or_in_place(out, dtype, a.gate, a.dtype, a.gate_stride, a.C, rows);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_gated_scan_workspace_bytes(const gdn_scan_args* args) {
  ScanProblem p;
  return scan_check(args, &p) == GDN_OK ? scan_fwd_workspace(p) : 0;
}

int gdn_gated_scan_fwd(const gdn_scan_args* args, void* ws, size_t ws_bytes, void* stream) {
  ScanProblem p;
  int st = scan_check(args, &p);
  if (st == GDN_OK) st = scan_pointers(p.a);
  if (st != GDN_OK) return st;
  const gdn_scan_args& a = p.a;
  if (!rows_ok(a.h, a.T) || !aligned16(a.h0) || !aligned16(a.h_final) || !aligned16(a.checkpoints)) return GDN_ERR_ARG;
  if (!scan_rows_apart(a, a.h)) return GDN_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, scan_fwd_workspace(p))) return GDN_ERR_WORKSPACE;
  if (a.T == 0 && (a.h_final == nullptr || a.h_final == a.h0)) return GDN_OK;
  return hip_status(launch_scan_fwd(p, ws, stream));
}

int gdn_gated_scan_step(const gdn_scan_args* args, float* state_inout, void* stream) {
  ScanProblem p;
  int st = scan_check(args, &p);
  if (st == GDN_OK) st = scan_pointers(p.a);
  if (st != GDN_OK) return st;
  if (!rows_ok(p.a.h, p.a.T) || state_inout == nullptr || !aligned16(state_inout) || !scan_rows_apart(p.a, p.a.h))
    return GDN_ERR_ARG;
  if (p.a.T == 0) return GDN_OK;
  return hip_status(launch_scan_step(p, state_inout, state_inout, stream));
}

size_t gdn_gated_scan_bwd_workspace_bytes(const gdn_scan_args* args) {
  ScanProblem p;
  return scan_check(args, &p) == GDN_OK ? scan_bwd_workspace(p) : 0;
}

int gdn_gated_scan_bwd(const gdn_scan_args* args, const void* d_h, const float* d_h_final, const gdn_scan_grads* grads,
                       void* ws, size_t ws_bytes, void* stream) {
  ScanProblem p;
  int st = scan_check(args, &p);
  if (st == GDN_OK) st = scan_pointers(p.a);
  if (st != GDN_OK) return st;
  const gdn_scan_args& a = p.a;
  if (grads == nullptr || !rows_ok(d_h, a.T) || !aligned16(d_h_final) || !aligned16(a.h0) || !aligned16(a.checkpoints))
    return GDN_ERR_ARG;
  if (!rows_ok(grads->dx, a.T) || !rows_ok(grads->df, a.T)) return GDN_ERR_ARG;
  if (a.i != nullptr ? !rows_ok(grads->di, a.T) : grads->di != nullptr) return GDN_ERR_ARG;
  if (!aligned16(grads->ddecay) || !aligned16(grads->dh0)) return GDN_ERR_ARG;
  if (a.gate != GDN_SCAN_POWER && grads->ddecay != nullptr) return GDN_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, scan_bwd_workspace(p))) return GDN_ERR_WORKSPACE;
  for (const void* out : {grads->dx, grads->df, grads->di})
    if (!scan_rows_apart(a, out) || !apart_or_in_place(out, a.dtype, d_h, a.dtype, a.C, a.C, a.B * a.T)) return GDN_ERR_ARG;
  // one segment's workgroup writes dh0, others may still read d_h_final
  const int64_t state = a.B * a.C * int64_t(sizeof(float));
  if (meets(grads->dh0, state, d_h_final, 1, state, state)) return GDN_ERR_ARG;
  if (a.T == 0 && grads->dh0 == nullptr && grads->ddecay == nullptr) return GDN_OK;
  return hip_status(launch_scan_bwd(p, d_h, d_h_final, *grads, ws, stream));
}

int gdn_short_conv_fwd(const gdn_conv_args* args, void* stream) {
  ConvProblem p;
  int st = conv_check(args, &p);
  if (st == GDN_OK) st = conv_pointers(p.a);
  if (st != GDN_OK) return st;
  const gdn_conv_args& a = p.a;
  if (!rows_ok(a.y, a.T) || !aligned16(a.s0) || !aligned16(a.s_final) || !conv_rows_apart(a)) return GDN_ERR_ARG;
  if (a.T == 0 && (a.s_final == nullptr || a.s_final == a.s0)) return GDN_OK;
  return hip_status(launch_conv_fwd(p, a.s0, a.s_final, stream));
}

int gdn_short_conv_step(const gdn_conv_args* args, void* state_inout, void* stream) {
  ConvProblem p;
  int st = conv_check(args, &p);
  if (st == GDN_OK) st = conv_pointers(p.a);
  if (st != GDN_OK) return st;
  if (!rows_ok(p.a.y, p.a.T) || state_inout == nullptr || !aligned16(state_inout) || !conv_rows_apart(p.a))
    return GDN_ERR_ARG;
  if (p.a.T == 0) return GDN_OK;
  return hip_status(launch_conv_fwd(p, state_inout, state_inout, stream));
}

size_t gdn_short_conv_bwd_workspace_bytes(const gdn_conv_args* args) {
  ConvProblem p;
  return conv_check(args, &p) == GDN_OK ? conv_bwd_workspace(p) : 0;
}

int gdn_short_conv_bwd(const gdn_conv_args* args, const void* d_y, const void* d_s_final, const gdn_conv_grads* grads,
                       void* ws, size_t ws_bytes, void* stream) {
  ConvProblem p;
  int st = conv_check(args, &p);
  if (st == GDN_OK) st = conv_pointers(p.a);
  if (st != GDN_OK) return st;
  const gdn_conv_args& a = p.a;
  if (grads == nullptr || !rows_ok(d_y, a.T) || !aligned16(d_s_final) || !aligned16(a.s0)) return GDN_ERR_ARG;
  if (!rows_ok(grads->dx, a.T) || !aligned16(grads->ds0) || !aligned4(grads->dw) || !aligned4(grads->dbias))
    return GDN_ERR_ARG;
  if (a.bias == nullptr && grads->dbias != nullptr) return GDN_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, conv_bwd_workspace(p))) return GDN_ERR_WORKSPACE;
  // a run reads rows of x and d_y, and of d_s_final, behind those whose gradients others write
  const int64_t rows = a.B * a.T, width = a.C * size_of(a.dtype), state = a.B * (a.W - 1) * width;
  if (meets(grads->dx, rows * width, a.x, rows, width, a.x_stride * size_of(a.dtype)) ||
      meets(grads->dx, rows * width, d_y, 1, rows * width, rows * width) ||
      meets(grads->ds0, state, a.s0, 1, state, state) || meets(grads->ds0, state, d_s_final, 1, state, state))
    return GDN_ERR_ARG;
  if (a.T == 0 && grads->ds0 == nullptr && grads->dw == nullptr && grads->dbias == nullptr) return GDN_OK;
  return hip_status(launch_conv_bwd(p, d_y, d_s_final, *grads, ws, stream));
}

int gdn_block_norm_fwd(const gdn_block_norm_args* args, void* stream) {
  BlockNormProblem p;
  int st = norm_check(args, &p);
  if (st == GDN_OK) st = norm_pointers(p.a);
  if (st != GDN_OK) return st;
  const gdn_block_norm_args& a = p.a;
  if (a.T == 0) return GDN_OK;
  if ((a.out == nullptr && a.residual_out == nullptr) || a.out == a.residual_out) return GDN_ERR_ARG;
  if (!aligned16(a.out) || !aligned16(a.residual_out)) return GDN_ERR_ARG;
  if (!norm_rows_apart(a, p.tokens, a.out, a.dtype) || !norm_rows_apart(a, p.tokens, a.residual_out, a.residual_dtype))
    return GDN_ERR_ARG;
  const int64_t all = p.tokens * a.C, bytes = all * size_of(a.residual_dtype);
  if (meets(a.out, all * size_of(a.dtype), a.residual_out, 1, bytes, bytes)) return GDN_ERR_ARG;
  return hip_status(launch_block_norm_fwd(p, stream));
}

size_t gdn_block_norm_bwd_workspace_bytes(const gdn_block_norm_args* args) {
  BlockNormProblem p;
  return norm_check(args, &p) == GDN_OK ? block_norm_bwd_workspace(p) : 0;
}

int gdn_block_norm_bwd(const gdn_block_norm_args* args, const gdn_block_norm_grads* g, void* ws, size_t ws_bytes,
                       void* stream) {
  BlockNormProblem p;
  int st = norm_check(args, &p);
  if (st == GDN_OK) st = norm_pointers(p.a);
  if (st != GDN_OK) return st;
  const gdn_block_norm_args& a = p.a;
  if (g == nullptr) return GDN_ERR_ARG;
  if (a.T > 0 && g->d_out == nullptr && g->d_residual_out == nullptr) return GDN_ERR_ARG;
  for (const void* x : {g->d_out, g->d_residual_out, (const void*)g->dr, (const void*)g->dy, (const void*)g->dgate})
    if (!aligned16(x)) return GDN_ERR_ARG;
  if (!aligned4(g->dscale) || !aligned4(g->dpost_weight) || !aligned4(g->dweight)) return GDN_ERR_ARG;
  if ((a.y == nullptr && a.T > 0 && g->dy != nullptr) || (a.gate == nullptr && a.T > 0 && g->dgate != nullptr) ||
      (a.scale == nullptr && g->dscale != nullptr) || (a.post_weight == nullptr && g->dpost_weight != nullptr) ||
      (a.weight == nullptr && g->dweight != nullptr))
    return GDN_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, block_norm_bwd_workspace(p))) return GDN_ERR_WORKSPACE;
  for (const auto& [out, dtype] : {std::pair<void*, int>{g->dr, a.residual_dtype}, {g->dy, a.dtype}, {g->dgate, a.dtype}}) {
    if (!norm_rows_apart(a, p.tokens, out, dtype) ||
        !apart_or_in_place(out, dtype, g->d_out, a.dtype, a.C, a.C, p.tokens) ||
        !apart_or_in_place(out, dtype, g->d_residual_out, a.residual_dtype, a.C, a.C, p.tokens))
      return GDN_ERR_ARG;
  }
  if (a.T == 0 && g->dscale == nullptr && g->dpost_weight == nullptr && g->dweight == nullptr) return GDN_OK;
  return hip_status(launch_block_norm_bwd(p, *g, ws, stream));
}

}  // extern "C"
