// Internal declarations of the operators around the delta rule: linear attention with a
// decay a head, the norms of queries and keys, and the gated norm.
#pragma once

#include <cstddef>
#include <cstdint>

#include "gdn.h"

namespace gdn {

// Linear attention after validation: strides resolved.
struct LinearProblem {
  int64_t B, T, H, Hk, dk, dv;
  int64_t group;              // value heads a key head serves
  int64_t ldq, ldk, ldv;      // elements from token to token
  int dtype;
  const void* q;
  const void* k;
  const void* v;
  const float* log_decay;
  const int32_t* seq_lens;
  const float* s0;
  float* s_final;
  void* o;
};

struct LinearGrads {
  const void* d_o;
  const float* d_s_final;
  void* dq;
  void* dk;
  void* dv;
  float* ds0;
};

// Rows of a norm: [tokens][heads][d] with `ld` elements from token to token.
struct QkNormProblem {
  gdn_qk_norm_args a;  // strides resolved
  int64_t tokens;      // B * T
};
struct GatedNormProblem {
  gdn_gated_norm_args a;
  int64_t tokens;
};

// Partial sums of weight gradients: at most this many blocks, one row of floats each (four
// blocks a CU; q / k norm gradients at 8,192 x 24 rows of 128: 512, 768, 2048 blocks 46, 40,
// 40 us against 38).
constexpr int64_t kNormPartials = 1024;

// Launchers (the .hip translation units); each returns a hipError_t as int.
int launch_linear_step(const LinearProblem& p, float* state, void* stream);
int launch_linear_fwd(const LinearProblem& p, void* ws, void* stream);
size_t linear_fwd_workspace(const LinearProblem& p);
int launch_linear_bwd(const LinearProblem& p, const LinearGrads& g, void* ws, void* stream);
size_t linear_bwd_workspace(const LinearProblem& p);
int launch_qk_norm_fwd(const QkNormProblem& p, void* stream);
int launch_qk_norm_bwd(const QkNormProblem& p, const gdn_qk_norm_grads& g, void* ws, void* stream);
int launch_gated_norm_fwd(const GatedNormProblem& p, void* stream);
int launch_gated_norm_bwd(const GatedNormProblem& p, const gdn_gated_norm_grads& g, void* ws, void* stream);

}  // namespace gdn
