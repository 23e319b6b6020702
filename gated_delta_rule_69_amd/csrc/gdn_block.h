// Internal declarations of the operators of a block: the gated recurrence a channel, the
// short convolution before it, and the norms around it.
#pragma once

#include <cstddef>
#include <cstdint>

#include "gdn.h"

namespace gdn {

// Arguments after validation: strides resolved (never 0).
struct ScanProblem {
  gdn_scan_args a;
};
struct ConvProblem {
  gdn_conv_args a;
};
struct BlockNormProblem {
  gdn_block_norm_args a;
  int64_t tokens;  // B * T
};

// Launchers (the .hip translation units); each returns a hipError_t as int.
size_t scan_fwd_workspace(const ScanProblem& p);
int launch_scan_fwd(const ScanProblem& p, void* ws, void* stream);
int launch_scan_step(const ScanProblem& p, const float* before, float* after, void* stream);
size_t scan_bwd_workspace(const ScanProblem& p);
int launch_scan_bwd(const ScanProblem& p, const void* d_h, const float* d_h_final, const gdn_scan_grads& g, void* ws,
                    void* stream);

// Tokens up to which a convolution always goes one by one, so that y may be x.
constexpr int64_t kConvInPlace = 8;
int launch_conv_fwd(const ConvProblem& p, const void* s0, void* s_final, void* stream);
size_t conv_bwd_workspace(const ConvProblem& p);
int launch_conv_bwd(const ConvProblem& p, const void* d_y, const void* d_s_final, const gdn_conv_grads& g, void* ws,
                    void* stream);

int launch_block_norm_fwd(const BlockNormProblem& p, void* stream);
size_t block_norm_bwd_workspace(const BlockNormProblem& p);
int launch_block_norm_bwd(const BlockNormProblem& p, const gdn_block_norm_grads& g, void* ws, void* stream);

}  // namespace gdn
