// Chunked passes of linear attention on float32 rows.
#include "gdn_linear_pass.h"

namespace gdn {

int launch_pass_f32(const LinearPasses& s, int count, int64_t B, int da, int dc, bool out, void* stream) {
  return launch_pass_any<float, float>(s, count, B, da, dc, out, static_cast<hipStream_t>(stream));
}

}  // namespace gdn
