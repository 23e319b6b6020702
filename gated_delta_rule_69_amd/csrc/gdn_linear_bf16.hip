// Chunked passes of linear attention on bf16 rows.
#include "gdn_linear_pass.h"

namespace gdn {

int launch_pass_bf16(const LinearPass& s, int64_t B, int da, int dc, bool rev, bool out, bool wide_out, void* stream) {
  hipStream_t hs = static_cast<hipStream_t>(stream);
  return wide_out ? launch_pass_any<__bf16, float>(s, B, da, dc, rev, out, hs)
                  : launch_pass_any<__bf16, __bf16>(s, B, da, dc, rev, out, hs);
}

}  // namespace gdn
