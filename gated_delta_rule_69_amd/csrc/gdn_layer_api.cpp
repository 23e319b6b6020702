// C ABI entry points of linear attention, the q / k norms and the gated norm: argument
// checks and dispatch. No HIP call here; launches live in the .hip files.
#include <cmath>

#include "gdn_layer.h"

namespace gdn {
namespace {

bool head_dim_ok(int64_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dtype_ok(int d) { return d == GDN_DTYPE_F32 || d == GDN_DTYPE_BF16; }

// Sizes: every element offset stays far inside int64, every grid inside 31 bits.
int sizes(int64_t B, int64_t T, int64_t H) {
  if (B < 1 || T < 0 || H < 1) return GDN_ERR_ARG;
  if (B > (1 << 20) || H > (1 << 16) || T > (int64_t(1) << 31)) return GDN_ERR_UNSUPPORTED;
  if (B * H > (1 << 24) || B * T > (int64_t(1) << 36)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// A token stride: 0 means contiguous; else at least a token's heads, in 16-byte steps.
int stride(int64_t given, int64_t heads, int64_t d, int dtype, int64_t* out) {
  const int64_t least = heads * d, step = dtype == GDN_DTYPE_BF16 ? 8 : 4;
  *out = given == 0 ? least : given;
  if (*out < least || *out % step != 0) return GDN_ERR_ARG;
  if (*out > (int64_t(1) << 24)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

bool ws_ok(const void* ws, size_t bytes, size_t need) {
  return ws != nullptr && bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

// Shapes of a linear-attention call; the pointers are copied unchecked.
int linear_shapes(const gdn_linear_args* a, LinearProblem* p) {
  if (a == nullptr || !dtype_ok(a->dtype) || a->reserved != 0) return GDN_ERR_ARG;
  int st = sizes(a->B, a->T, a->H);
  if (st != GDN_OK) return st;
  if (a->Hk < 1 || a->Hk > a->H || a->H % a->Hk != 0) return GDN_ERR_ARG;
  if (a->T > (int64_t(1) << 31) - (1 << 16)) return GDN_ERR_UNSUPPORTED;  // positions are ints, a chunk's end included
  if (!head_dim_ok(a->dk) || !head_dim_ok(a->dv)) return GDN_ERR_UNSUPPORTED;
  // a launch has fewer than 2^32 threads: four for each of a head's channels
  if (a->B * a->H * (a->dk > a->dv ? a->dk : a->dv) >= int64_t(1) << 30) return GDN_ERR_UNSUPPORTED;
  *p = LinearProblem{};
  if ((st = stride(a->q_stride, a->Hk, a->dk, a->dtype, &p->ldq)) != GDN_OK) return st;
  if ((st = stride(a->k_stride, a->Hk, a->dk, a->dtype, &p->ldk)) != GDN_OK) return st;
  if ((st = stride(a->v_stride, a->H, a->dv, a->dtype, &p->ldv)) != GDN_OK) return st;
  p->B = a->B, p->T = a->T, p->H = a->H, p->Hk = a->Hk, p->dk = a->dk, p->dv = a->dv;
  p->group = a->H / a->Hk;
  p->dtype = a->dtype;
  p->q = a->q, p->k = a->k, p->v = a->v, p->log_decay = a->log_decay, p->seq_lens = a->seq_lens;
  p->s0 = a->s0, p->s_final = a->s_final, p->o = a->o;
  return GDN_OK;
}

// Pointers every linear entry point reads; arrays of no tokens may be NULL.
int linear_pointers(const LinearProblem& p) {
  auto need = [&](const void* x) { return p.T == 0 ? aligned16(x) : (x != nullptr && aligned16(x)); };
  if (!need(p.q) || !need(p.k) || !need(p.v)) return GDN_ERR_ARG;
  if (p.log_decay == nullptr || !aligned4(p.log_decay) || !aligned4(p.seq_lens)) return GDN_ERR_ARG;
  return GDN_OK;
}

int qk_norm_check(const gdn_qk_norm_args* a, QkNormProblem* p) {
  if (a == nullptr || !dtype_ok(a->dtype) || a->reserved != 0) return GDN_ERR_ARG;
  if (a->norm != GDN_NORM_RMS && a->norm != GDN_NORM_L2) return GDN_ERR_ARG;
  if (a->interleaved != 0 && a->interleaved != 1) return GDN_ERR_ARG;
  if (!(a->eps >= 0.0f) || !std::isfinite(a->q_scale)) return GDN_ERR_ARG;
  int st = sizes(a->B, a->T, a->Hq);
  if (st == GDN_OK) st = sizes(a->B, a->T, a->Hk);
  if (st != GDN_OK) return st;
  if (!head_dim_ok(a->d)) return GDN_ERR_UNSUPPORTED;
  if (a->rot < 0 || a->rot > a->d || a->rot % 8 != 0) return GDN_ERR_ARG;
  p->a = *a;
  if ((st = stride(a->q_stride, a->Hq, a->d, a->dtype, &p->a.q_stride)) != GDN_OK) return st;
  if ((st = stride(a->k_stride, a->Hk, a->d, a->dtype, &p->a.k_stride)) != GDN_OK) return st;
  p->tokens = a->B * a->T;
  return GDN_OK;
}

int qk_norm_pointers(const QkNormProblem& p) {
  const gdn_qk_norm_args& a = p.a;
  auto need = [&](const void* x) { return a.T == 0 ? aligned16(x) : (x != nullptr && aligned16(x)); };
  if (!need(a.q) || !need(a.k) || !aligned16(a.wq) || !aligned16(a.wk)) return GDN_ERR_ARG;
  if (a.rot > 0 && a.T > 0) {
    if (!need(a.cos) || !need(a.sin) || !aligned4(a.positions)) return GDN_ERR_ARG;
    if (a.n_pos < 1 || (a.positions == nullptr && a.n_pos < a.T)) return GDN_ERR_ARG;
    if (a.n_pos > (int64_t(1) << 31)) return GDN_ERR_UNSUPPORTED;
  }
  return GDN_OK;
}

int gated_norm_check(const gdn_gated_norm_args* a, GatedNormProblem* p) {
  if (a == nullptr || !dtype_ok(a->dtype) || a->reserved != 0) return GDN_ERR_ARG;
  if (a->activation != GDN_ACT_SILU && a->activation != GDN_ACT_SIGMOID) return GDN_ERR_ARG;
  if (!(a->eps >= 0.0f)) return GDN_ERR_ARG;
  int st = sizes(a->B, a->T, a->H);
  if (st != GDN_OK) return st;
  if (!head_dim_ok(a->d)) return GDN_ERR_UNSUPPORTED;
  p->a = *a;
  if ((st = stride(a->x_stride, a->H, a->d, a->dtype, &p->a.x_stride)) != GDN_OK) return st;
  if ((st = stride(a->gate_stride, a->H, a->d, a->dtype, &p->a.gate_stride)) != GDN_OK) return st;
  p->tokens = a->B * a->T;
  return GDN_OK;
}

int gated_norm_pointers(const GatedNormProblem& p) {
  const gdn_gated_norm_args& a = p.a;
  auto need = [&](const void* x) { return a.T == 0 ? aligned16(x) : (x != nullptr && aligned16(x)); };
  return need(a.x) && need(a.gate) && aligned16(a.weight) ? GDN_OK : GDN_ERR_ARG;
}

int hip_status(int rc) { return rc == 0 ? GDN_OK : GDN_ERR_HIP; }

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_linear_workspace_bytes(const gdn_linear_args* args) {
  LinearProblem p;
  return linear_shapes(args, &p) == GDN_OK ? linear_fwd_workspace(p) : 0;
}

int gdn_linear_chunk_fwd(const gdn_linear_args* args, void* ws, size_t ws_bytes, void* stream) {
  LinearProblem p;
  int st = linear_shapes(args, &p);
  if (st == GDN_OK) st = linear_pointers(p);
  if (st != GDN_OK) return st;
  if ((p.T > 0 && p.o == nullptr) || !aligned16(p.o) || !aligned16(p.s0) || !aligned16(p.s_final))
    return GDN_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, linear_fwd_workspace(p))) return GDN_ERR_WORKSPACE;
  if (p.T == 0 && (p.s_final == nullptr || p.s_final == p.s0)) return GDN_OK;
  return hip_status(launch_linear_fwd(p, ws, stream));
}

int gdn_linear_recurrent_step(const gdn_linear_args* args, float* state_inout, void* stream) {
  LinearProblem p;
  int st = linear_shapes(args, &p);
  if (st == GDN_OK) st = linear_pointers(p);
  if (st != GDN_OK) return st;
  if ((p.T > 0 && p.o == nullptr) || !aligned16(p.o)) return GDN_ERR_ARG;
  if (state_inout == nullptr || !aligned16(state_inout)) return GDN_ERR_ARG;
  if (p.T == 0) return GDN_OK;
  return hip_status(launch_linear_step(p, state_inout, stream));
}

size_t gdn_linear_bwd_workspace_bytes(const gdn_linear_args* args) {
  LinearProblem p;
  return linear_shapes(args, &p) == GDN_OK ? linear_bwd_workspace(p) : 0;
}

int gdn_linear_chunk_bwd(const gdn_linear_args* args, const void* d_o, const float* d_s_final,
                         const gdn_linear_grads* grads, void* ws, size_t ws_bytes, void* stream) {
  LinearProblem p;
  int st = linear_shapes(args, &p);
  if (st == GDN_OK) st = linear_pointers(p);
  if (st != GDN_OK) return st;
  if (grads == nullptr) return GDN_ERR_ARG;
  auto need = [&](const void* x) { return p.T == 0 ? aligned16(x) : (x != nullptr && aligned16(x)); };
  if (!need(d_o) || !need(grads->dq) || !need(grads->dk) || !need(grads->dv)) return GDN_ERR_ARG;
  if (!aligned16(p.s0) || !aligned16(d_s_final) || !aligned16(grads->ds0)) return GDN_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, linear_bwd_workspace(p))) return GDN_ERR_WORKSPACE;
  if (p.T == 0 && grads->ds0 == nullptr) return GDN_OK;
  const LinearGrads g{d_o, d_s_final, grads->dq, grads->dk, grads->dv, grads->ds0};
  return hip_status(launch_linear_bwd(p, g, ws, stream));
}

int gdn_qk_norm_fwd(const gdn_qk_norm_args* args, void* stream) {
  QkNormProblem p;
  int st = qk_norm_check(args, &p);
  if (st == GDN_OK) st = qk_norm_pointers(p);
  if (st != GDN_OK) return st;
  const gdn_qk_norm_args& a = p.a;
  if (a.T == 0) return GDN_OK;
  if (a.q_out == nullptr || !aligned16(a.q_out) || a.k_out == nullptr || !aligned16(a.k_out)) return GDN_ERR_ARG;
  // in place only row over row
  if (a.q_out == a.q && a.q_stride != a.Hq * a.d) return GDN_ERR_ARG;
  if (a.k_out == a.k && a.k_stride != a.Hk * a.d) return GDN_ERR_ARG;
  return hip_status(launch_qk_norm_fwd(p, stream));
}

size_t gdn_qk_norm_bwd_workspace_bytes(const gdn_qk_norm_args* args) {
  QkNormProblem p;
  if (qk_norm_check(args, &p) != GDN_OK) return 0;
  return size_t(kNormPartials) * size_t(p.a.d) * 2 * sizeof(float);
}

int gdn_qk_norm_bwd(const gdn_qk_norm_args* args, const gdn_qk_norm_grads* g, void* ws, size_t ws_bytes,
                    void* stream) {
  QkNormProblem p;
  int st = qk_norm_check(args, &p);
  if (st == GDN_OK) st = qk_norm_pointers(p);
  if (st != GDN_OK) return st;
  const gdn_qk_norm_args& a = p.a;
  if (g == nullptr || g->reserved != 0) return GDN_ERR_ARG;
  if (g->grad_dtype != GDN_DTYPE_F32 && g->grad_dtype != a.dtype) return GDN_ERR_ARG;
  auto need = [&](const void* x) { return a.T == 0 ? aligned16(x) : (x != nullptr && aligned16(x)); };
  if (!need(g->dq_out) || !need(g->dk_out) || !need(g->dq) || !need(g->dk)) return GDN_ERR_ARG;
  if (!aligned4(g->dwq) || !aligned4(g->dwk)) return GDN_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, gdn_qk_norm_bwd_workspace_bytes(args))) return GDN_ERR_WORKSPACE;
  if (a.T == 0 && g->dwq == nullptr && g->dwk == nullptr) return GDN_OK;
  return hip_status(launch_qk_norm_bwd(p, *g, ws, stream));
}

int gdn_gated_norm_fwd(const gdn_gated_norm_args* args, void* stream) {
  GatedNormProblem p;
  int st = gated_norm_check(args, &p);
  if (st == GDN_OK) st = gated_norm_pointers(p);
  if (st != GDN_OK) return st;
  const gdn_gated_norm_args& a = p.a;
  if (a.T == 0) return GDN_OK;
  if (a.y == nullptr || !aligned16(a.y)) return GDN_ERR_ARG;
  if (a.y == a.x && a.x_stride != a.H * a.d) return GDN_ERR_ARG;
  if (a.y == a.gate && a.gate_stride != a.H * a.d) return GDN_ERR_ARG;
  return hip_status(launch_gated_norm_fwd(p, stream));
}

size_t gdn_gated_norm_bwd_workspace_bytes(const gdn_gated_norm_args* args) {
  GatedNormProblem p;
  if (gated_norm_check(args, &p) != GDN_OK) return 0;
  return size_t(kNormPartials) * size_t(p.a.d) * sizeof(float);
}

int gdn_gated_norm_bwd(const gdn_gated_norm_args* args, const gdn_gated_norm_grads* g, void* ws,
                       size_t ws_bytes, void* stream) {
  GatedNormProblem p;
  int st = gated_norm_check(args, &p);
  if (st == GDN_OK) st = gated_norm_pointers(p);
  if (st != GDN_OK) return st;
  const gdn_gated_norm_args& a = p.a;
  if (g == nullptr) return GDN_ERR_ARG;
  auto need = [&](const void* x) { return a.T == 0 ? aligned16(x) : (x != nullptr && aligned16(x)); };
  if (!need(g->dy) || !need(g->dx) || !need(g->dgate) || !aligned4(g->dweight)) return GDN_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, gdn_gated_norm_bwd_workspace_bytes(args))) return GDN_ERR_WORKSPACE;
  if (a.T == 0 && g->dweight == nullptr) return GDN_OK;
  return hip_status(launch_gated_norm_bwd(p, *g, ws, stream));
}

}  // extern "C"
