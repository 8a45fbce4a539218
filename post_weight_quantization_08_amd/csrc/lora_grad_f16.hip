// The adapters' gradients for f16 factors.
#include "lora_grad_kernels.h"

namespace gq {

void grad_launch_f16(const GradArgs& a, bool codes, bool wide, int64_t max_chunks, GradStage stage, hipStream_t st) {
  grad_launch<GPTQ_F16>(a, codes, wide, max_chunks, stage, st);
}

}  // namespace gq
