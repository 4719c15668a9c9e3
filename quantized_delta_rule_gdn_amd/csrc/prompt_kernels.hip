// prompt_kernels.hip -- gfx950 kernels of the chunked prompt forms.
#include "prompt_common.h"

namespace damp {

int64_t prefill_ws_bytes(bool delta, int d, int decay, int bf16, int32_t B, int32_t T, int32_t H) { return 0; }

hipError_t launch_prefill(bool delta, int d, int decay, int bf16, const PromptArgs& a, hipStream_t s) {
  return launch_prompt_token(d, delta, decay, bf16, a, s);
}

}  // namespace damp
