// The gated recurrence a channel: its bfloat16 kernels (a translation unit of their own so that
// the instances compile side by side).
#include "gdn_scan_pass.h"

namespace gdn {
namespace scan {
int step_bf16(const ScanProblem& q, const Pass& p, hipStream_t s) { return launch_step<__bf16>(q, p, s); }
int fwd_bf16(const ScanProblem& q, const Pass& p, hipStream_t s) { return launch_pass<__bf16, false>(q, p, s); }
int bwd_bf16(const ScanProblem& q, const Pass& p, hipStream_t s) { return launch_pass<__bf16, true>(q, p, s); }
}  // namespace scan
}  // namespace gdn
