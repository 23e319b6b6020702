// The gated recurrence a channel: its float32 kernels (a translation unit of their own so that
// the instances compile side by side).
#include "gdn_scan_pass.h"

namespace gdn {
namespace scan {
int step_f32(const ScanProblem& q, const Pass& p, hipStream_t s) { return launch_step<float>(q, p, s); }
int fwd_f32(const ScanProblem& q, const Pass& p, hipStream_t s) { return launch_pass<float, false>(q, p, s); }
int bwd_f32(const ScanProblem& q, const Pass& p, hipStream_t s) { return launch_pass<float, true>(q, p, s); }
}  // namespace scan
}  // namespace gdn
