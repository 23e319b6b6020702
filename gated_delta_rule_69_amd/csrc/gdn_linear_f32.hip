// Chunked passes of linear attention on float32 rows.
#include "gdn_linear_pass.h"

namespace gdn {

int launch_pass_f32(const LinearPass& s, int64_t B, int da, int dc, bool rev, bool out, void* stream) {
  return launch_pass_any<float, float>(s, B, da, dc, rev, out, static_cast<hipStream_t>(stream));
}

}  // namespace gdn
