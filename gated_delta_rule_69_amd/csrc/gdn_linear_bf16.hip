// Chunked passes of linear attention on bf16 rows.
#include "gdn_linear_pass.h"

namespace gdn {

int launch_pass_bf16(const LinearPasses& s, int count, int64_t B, int da, int dc, bool out, bool wide_out, void* stream) {
  hipStream_t hs = static_cast<hipStream_t>(stream);
  return wide_out ? launch_pass_any<__bf16, float>(s, count, B, da, dc, out, hs)
                  : launch_pass_any<__bf16, __bf16>(s, count, B, da, dc, out, hs);
}

}  // namespace gdn
